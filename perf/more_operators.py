"""Cases of the block-scaled cache, of draft verification and of the page operators, in plain
PyTorch and through the library.

Operators of a serving loop over paged K/V pools ([num_pages, Hkv, page_size, 128]):

* ``append``   rotary positions on the new queries and keys, and the new keys and values
               written to a cache of e4m3 codes with one scale per block of tokens and head;
* ``attn``     causal attention of each request's newest tokens over such a cache;
* ``verify``   drafted tokens accepted or rejected by the target's probabilities and given
               random numbers, and the token that follows the accepted ones;
* ``fork``     rows of the slot table forked: full pages shared, the last one copied, after
               the last pass's children were freed;
* ``compact``  the live pages of scattered pools moved to their front.

``listed`` holds the cases, ``draw`` more of the same ranges, ``run`` one pass: through
elementary torch operations, or, where ``own`` is set, through the library.
"""

import math
import random

import torch

own = False

HEAD_DIM = 128
SM_SCALE = float(torch.tensor(HEAD_DIM ** -0.5, dtype=torch.float32))
ROPE_BASE = 10000.0
CODE_MAX = 448.0  # of e4m3
UNITS = 2.0 ** 42  # of a weight that a token is sampled by


def listed():
    return [
        # one new token for each of 32 decoding requests (what is cached does not count): launch
        # latency
        dict(name="append_decode_32", op="append", bs=32, ctx=200, ragged=False, new=1, hq=32,
             hkv=8, page=64, block=64, rot=128, interleaved=False),
        # the last chunk of a prompt entering the cache
        dict(name="append_prompt_8k", op="append", bs=1, ctx=8192, ragged=False, new=8192, hq=32,
             hkv=8, page=64, block=64, rot=128, interleaved=False),
        # one request decoding: latency
        dict(name="attn_bs1_1k", op="attn", bs=1, ctx=1024, ragged=False, new=1, hq=32, hkv=8,
             page=64, block=64),
        # a ragged batch verifying chains of up to five tokens, 5 heads to a kv head, small
        # pages and blocks, odd lengths
        dict(name="attn_bs8_chain", op="attn", bs=8, ctx=4001, ragged=True, new=5, hq=40, hkv=8,
             page=16, block=16),
        # the serving batch: 32 requests at 8K tokens
        dict(name="attn_bs32_8k", op="attn", bs=32, ctx=8192, ragged=False, new=1, hq=32, hkv=8,
             page=64, block=64),
        # the ragged batch up to 16K tokens, 64 heads
        dict(name="attn_bs64_ragged", op="attn", bs=64, ctx=16384, ragged=True, new=1, hq=64,
             hkv=8, page=64, block=32),
        # one request's chain of four drafted tokens
        dict(name="verify_bs1_chain", op="verify", bs=1, new=5, vocab=32000, tree=False),
        # the serving batch, eight drafted tokens each, a large vocabulary
        dict(name="verify_bs32_chain", op="verify", bs=32, new=9, vocab=128000, tree=False),
        # trees of the draft's likeliest tokens, an odd vocabulary
        dict(name="verify_bs16_tree", op="verify", bs=16, new=32, vocab=100003, tree=True),
        # one prompt of 8001 tokens answered four times: eight layers' last pages copied
        dict(name="fork_1x4", op="fork", bs=1, fan=4, ctx=8001, ragged=False, hkv=8, page=64,
             layers=8, kv="bf16"),
        # a batch of ragged prompts answered twice each
        dict(name="fork_32x2_ragged", op="fork", bs=32, fan=2, ctx=4001, ragged=True, hkv=8,
             page=64, layers=8, kv="e4m3"),
        # pools of 4096 pages, half of them live and scattered, four layers: a quarter moves
        dict(name="compact_4096", op="compact", bs=32, ctx=4096, ragged=False, hkv=8, page=64,
             layers=4, kv="bf16", spare=2048),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["append", "attn", "attn", "attn", "verify", "verify", "fork", "compact"])
        hkv = rng.choice([1, 2, 4, 5, 8, 16])
        page = rng.choice([16, 32, 64, 128])
        c = dict(op=op, bs=_log_int(rng, 1, 64))
        if op in ("append", "attn"):
            group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            c.update(ctx=_log_int(rng, 16, 16384), ragged=rng.random() < 0.5, hq=hkv * group,
                     hkv=hkv, page=page, block=rng.choice([b for b in (16, 32, 64, 128) if b <= page]))
            if op == "append":
                c.update(new=_log_int(rng, 1, c["ctx"]), rot=16 * rng.randint(1, 8),
                         interleaved=rng.random() < 0.5)
            else:
                c.update(new=rng.choice([1, 1, rng.randint(2, 16)]))
        elif op == "verify":
            c.update(new=rng.randint(1, 32), vocab=_log_int(rng, 1000, 160000),
                     tree=rng.random() < 0.5)
        else:
            c.update(ctx=_log_int(rng, 16, 8192), ragged=rng.random() < 0.5, hkv=hkv, page=page,
                     layers=rng.randint(1, 8), kv=rng.choice(["bf16", "e4m3"]))
            if op == "fork":
                c.update(fan=rng.randint(1, 4))
            else:
                c.update(spare=_log_int(rng, 1, 4096))
            size = 2 * c["layers"] * _page_bytes(c) * _pages(c)
            if size > 6e9:
                continue
        w = work(c)
        if op == "verify" and 8 * c["vocab"] * c["new"] * c["bs"] > 1.0e9:
            continue
        if op == "append" and sum(_new(c)) > 8192:
            continue
        # no more than the largest listed case of bytes and of products
        if w["bytes"] <= 2.1e9 and w["flops"] <= 2.0e10:
            return c


# ---- lengths: fixed by the case, so that its work does not depend on the seed -----------


def lengths(c):
    """Cached tokens of each request (new ones among them)."""
    if not c["ragged"]:
        return [c["ctx"]] * c["bs"]
    n = [max(1, (2 * i + 1) * c["ctx"] // (2 * c["bs"])) for i in range(c["bs"])]
    random.Random(c["bs"] * 100003 + c["ctx"]).shuffle(n)
    return n


def _new(c):
    """New tokens of each request: up to ``new``, no more than it has cached."""
    r = random.Random(c["bs"] * 7919 + c["new"])
    want = [r.randint(1, c["new"]) if c["ragged"] else c["new"] for _ in range(c["bs"])]
    return [min(a, b) for a, b in zip(want, lengths(c))]


def _pages(c):
    per = sum(-(-n // c["page"]) for n in lengths(c))
    return per + (c["bs"] * c["fan"] + 3 if c["op"] == "fork" else c.get("spare", 0))


def _page_bytes(c):
    """Of one pool (K or V), scales among them."""
    rows = c["hkv"] * c["page"] * HEAD_DIM
    return 2 * rows if c["kv"] == "bf16" else rows + 4 * c["hkv"]


def work(c):
    if c["op"] == "append":
        t, n = sum(_new(c)), lengths(c)
        blocks = sum(-(-x // c["block"]) - (x - d) // c["block"] for x, d in zip(n, _new(c)))
        return {"bytes": t * (c["hq"] * 512 + c["hkv"] * 768 + 8) + blocks * c["hkv"] * 8,
                "flops": 3 * t * (c["hq"] + c["hkv"]) * c["rot"] + 4 * t * c["hkv"] * HEAD_DIM}
    if c["op"] == "attn":
        n, d = lengths(c), _new(c)
        rows = sum(d) * c["hq"]
        pairs = sum(di * x - di * (di - 1) // 2 for di, x in zip(d, n)) * c["hq"]
        scales = sum(-(-x // c["block"]) for x in n) * c["hkv"] * 8
        return {"bytes": sum(n) * c["hkv"] * 256 + scales + rows * 516,
                "flops": 4 * HEAD_DIM * pairs}
    if c["op"] == "verify":
        # one row of the target's probabilities a request (and of the draft's) is summed
        rows = c["bs"] * (1 if c["tree"] or c["new"] == 1 else 2)
        return {"bytes": rows * c["vocab"] * 4 + c["bs"] * c["new"] * 24,
                "flops": 2 * rows * c["vocab"]}
    n = lengths(c)
    if c["op"] == "fork":
        full = sum(x // c["page"] for x in n) * c["fan"]
        copied = sum(1 for x in n if x % c["page"]) * c["fan"]
        table = 8 * full * c["page"] + 8 * full
        return {"bytes": 4 * c["layers"] * copied * _page_bytes(c) + table, "flops": full}
    used = sum(-(-x // c["page"]) for x in n)
    moved = used * c["spare"] // (used + c["spare"])  # of pages scattered evenly
    return {"bytes": 4 * c["layers"] * moved * _page_bytes(c) + 8 * (used + c["spare"]),
            "flops": used + c["spare"]}


# ---- inputs ---------------------------------------------------------------------------------


def _inverse_frequencies(rot):
    return ROPE_BASE ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)


def _codes(shape, g, spread):
    """Codes of normal values, saturated."""
    x = torch.randn(shape, generator=g, device="cuda").mul_(spread).clamp_(-CODE_MAX, CODE_MAX)
    return x.to(torch.float8_e4m3fn)


def _prepare_blocks(c, s, g):
    """A block-scaled cache of the requests, scattered over its pool, and their new rows."""
    dev = "cuda"
    n, d = lengths(c), _new(c)
    per = [-(-x // c["page"]) for x in n]
    total = sum(per) + 2
    order = torch.randperm(total, generator=g, device=dev, dtype=torch.int32)
    width = max(per)
    count = torch.tensor(per, device=dev)
    col = torch.arange(width, device=dev)
    at = (torch.cumsum(count, 0) - count)[:, None] + col
    s["page_table"] = torch.where(col < count[:, None], order[at.clamp(max=total - 1)], 0) \
        .to(torch.int32).contiguous()
    s["max_seq_pages"] = width
    s["cache_seqlens"] = torch.tensor(n, device=dev, dtype=torch.int32)
    s["cu_seqlens_q"] = torch.tensor([sum(d[:i]) for i in range(len(d) + 1)], device=dev,
                                     dtype=torch.int32)
    s["max_q_len"], rows = max(d), sum(d)
    shape = (total, c["hkv"], c["page"], HEAD_DIM)
    for x in "kv":
        s[x + "_cache"] = _codes(shape, g, 100.0)
    blocks = (total, c["hkv"], c["page"] // c["block"])
    if c["op"] == "attn":
        s["q"] = torch.randn((rows, c["hq"], HEAD_DIM), generator=g, device=dev,
                             dtype=torch.bfloat16)
        for x in "kv":
            s[x + "_scale"] = torch.rand(blocks, generator=g, device=dev) * 0.015 + 0.005
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((rows, c["hq"]), dtype=torch.float32, device=dev)
        return
    # what earlier appends left: powers of two, some of them too small for the new rows
    for x in "kv":
        s[x + "_scale"] = torch.exp2(-torch.randint(5, 9, blocks, generator=g, device=dev).float())
    qkv = torch.randn((rows, c["hq"] + 2 * c["hkv"], HEAD_DIM), generator=g, device=dev,
                      dtype=torch.bfloat16)  # one projection's output: q, k and v are views
    s["q"], s["k"], s["v"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
    first = torch.tensor([x - y for x, y in zip(n, d)], device=dev)
    request = torch.repeat_interleave(torch.arange(c["bs"], device=dev),
                                      torch.tensor(d, device=dev), output_size=rows)
    s["positions"] = torch.arange(rows, device=dev) - s["cu_seqlens_q"].long()[request] + \
        first[request]
    s["inv_freq"] = _inverse_frequencies(c["rot"]).to(dev)
    s["q_out"] = torch.empty((rows, c["hq"], HEAD_DIM), dtype=torch.bfloat16, device=dev)


def _trees(bs, new, r):
    """Parents (the node's index in its request) and ancestor masks of seeded trees."""
    parents, masks = [], []
    for _ in range(bs):
        here = []
        for i in range(new):
            parent = r.randint(max(0, i - 6), i - 1) if i else -1
            parents.append(parent)
            here.append((here[parent] if parent >= 0 else 0) | (1 << i))
        masks += here
    return parents, masks


def _prepare_verify(c, s, g, seed):
    dev, bs, new, vocab = "cuda", c["bs"], c["new"], c["vocab"]
    rows = bs * new
    x = torch.randn((rows, vocab), generator=g, device=dev).mul_(3.0)
    s["target_probs"] = torch.softmax(x, -1)
    node = torch.arange(rows, device=dev) % new
    if c["tree"]:
        parents, masks = _trees(bs, new, random.Random(seed))
        s["parents"] = torch.tensor(parents, device=dev, dtype=torch.int32)
        s["masks"] = torch.tensor(masks, device=dev).view(bs, new)
        s["draft_probs"] = None
        # the rank-th likeliest token of the draft's idea of the parent's row: siblings differ
        up = torch.arange(bs, device=dev).repeat_interleave(new) * new + s["parents"].clamp(min=0)
        rank = torch.zeros(rows, dtype=torch.long)
        seen = {}
        for i, p in enumerate(parents):
            key = (i // new, p)
            rank[i] = seen.get(key, 0)
            seen[key] = int(rank[i]) + 1
        x.add_(torch.randn(x.shape, generator=g, device=dev).mul_(0.3))
        best = torch.topk(x, min(32, vocab), dim=-1).indices
        s["tokens"] = best[up, rank.to(dev)]
    else:
        s["parents"] = None
        x.add_(torch.randn(x.shape, generator=g, device=dev).mul_(0.5))
        s["draft_probs"] = torch.softmax(x, -1)
        # row i holds what token i + 1 was drawn from
        at = torch.rand((rows, 1), generator=g, device=dev)
        drawn = (torch.cumsum(s["draft_probs"], -1) < at).sum(-1).clamp(max=vocab - 1)
        s["tokens"] = torch.where(node > 0, drawn.roll(1), 0).contiguous()
    s["uniforms"] = torch.rand((rows,), generator=g, device=dev)
    s["final_uniforms"] = torch.rand((bs,), generator=g, device=dev)
    s["cu_seqlens_q"] = torch.arange(0, rows + 1, new, device=dev, dtype=torch.int32)
    s["cache_seqlens"] = torch.randint(new, new + 8192, (bs,), generator=g, device=dev,
                                       dtype=torch.int32)
    s["kept"] = torch.empty((bs, new), dtype=torch.int32, device=dev)
    for name in ("counts", "begin"):
        s[name] = torch.empty((bs,), dtype=torch.int32, device=dev)
    s["next_tokens"] = torch.empty((bs,), dtype=torch.int64, device=dev)


def _prepare_pages(c, s, g):
    dev, page = "cuda", c["page"]
    n = lengths(c)
    per = [-(-x // page) for x in n]
    total = _pages(c)
    fan = c.get("fan", 0)
    rows = c["bs"] * (1 + fan)
    width = max(per)
    order = torch.randperm(total, generator=g, device=dev)
    count = torch.tensor(per, device=dev)
    col = torch.arange(width, device=dev)
    at = (torch.cumsum(count, 0) - count)[:, None] + col
    mine = col < count[:, None]
    pages = order[at.clamp(max=total - 1)]
    s["page_refs"] = torch.zeros(total, dtype=torch.int32, device=dev)
    s["page_refs"][pages[mine]] = 1
    slots = pages[..., None] * page + torch.arange(page, device=dev)
    table = torch.full((rows, width * page), -1, dtype=torch.int32, device=dev)
    table[:c["bs"]] = torch.where(mine[..., None], slots, -1).flatten(1).to(torch.int32)
    s["req_to_token"], s["max_seq_pages"] = table, width
    lens = torch.tensor(n, device=dev, dtype=torch.int32)
    if c["op"] == "fork":
        s["parents"] = torch.arange(c["bs"], device=dev).repeat_interleave(fan)
        s["children"] = c["bs"] + torch.randperm(c["bs"] * fan, generator=g, device=dev)
        s["lens"] = lens.repeat_interleave(fan).contiguous()
        s["child_lens"] = torch.empty_like(s["lens"])
    else:
        s["rows"], s["lens"] = torch.arange(c["bs"], device=dev), lens
        s["scattered"] = [table.clone(), s["page_refs"].clone()]
        s["page_map"] = torch.empty(total, dtype=torch.int32, device=dev)
        s["num_live"] = torch.empty(1, dtype=torch.int32, device=dev)
    s["pools"] = []
    shape = (total, c["hkv"], page, HEAD_DIM)
    for _ in range(2 * c["layers"]):
        if c["kv"] == "bf16":
            s["pools"].append(torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16))
        else:
            codes = torch.randint(0, 127, shape, generator=g, device=dev, dtype=torch.uint8)
            s["pools"].append(codes.view(torch.float8_e4m3fn))
            s["pools"].append(torch.rand((total, c["hkv"], 1), generator=g, device=dev))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] in ("append", "attn"):
        _prepare_blocks(case, s, g)
    elif case["op"] == "verify":
        _prepare_verify(case, s, g, seed)
    else:
        _prepare_pages(case, s, g)
    return s


# ---- the plain forms ------------------------------------------------------------------------


def _plain_append(s):
    c = s["case"]
    dev, page, block = s["q"].device, c["page"], c["block"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotated(x):
        x = x.float()
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else r.chunk(2, -1)
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((r, rest), -1)

    s["q_out"].copy_(rotated(s["q"]))
    cu = s["cu_seqlens_q"].long()
    t = torch.arange(s["q"].shape[0], device=dev)
    request = torch.searchsorted(cu, t, right=True) - 1
    count = cu[1:] - cu[:-1]
    at = s["cache_seqlens"].long()[request] - count[request] + t - cu[request]
    where, row = s["page_table"].long()[request, at // page], at % page
    blocks = page // block
    home = where * blocks + row // block  # each token's block
    total = s["k_cache"].shape[0] * blocks
    first = torch.full((total,), block, device=dev).scatter_reduce(0, home, row % block, "amin")
    for name, x in (("k", rotated(s["k"])), ("v", s["v"].float())):
        codes = s[name + "_cache"].view(torch.uint8).unflatten(2, (blocks, block))
        old = s[name + "_scale"].transpose(1, 2).reshape(total, -1)
        big = torch.zeros_like(old).scatter_reduce(
            0, home[:, None].expand(-1, c["hkv"]), x.abs().amax(-1), "amax")
        m, e = torch.frexp(big)  # big = m 2^e, m in [1/2, 1): the largest code is 7/8 2^9
        want = torch.ldexp(torch.ones_like(m), (e - 9 + (m > 0.875).int()).clamp(min=-126))
        want = torch.where(big > 0, want, 0.0)
        new = torch.where(first[:, None] == 0, want, torch.maximum(old, want))
        new = torch.where(first[:, None] < block, new, old)
        # the rows that a block held before take its new scale
        b = torch.unique(home)
        held = codes.transpose(1, 2)[b // blocks, b % blocks]  # [touched, Hkv, block, 128]
        ratio = torch.where(new[b] > 0, old[b] / new[b], 1.0)[..., None, None]
        again = (held.view(torch.float8_e4m3fn).float() * ratio).to(torch.float8_e4m3fn)
        stays = torch.arange(block, device=dev)[:, None] >= first[b][:, None, None, None]
        held = torch.where(stays | (ratio == 1), held, again.view(torch.uint8))
        codes.transpose(1, 2)[b // blocks, b % blocks] = held
        scale = new[home]
        y = x * torch.where(scale > 0, 1 / scale, 0.0)[..., None]
        y = y.clamp(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_cache"].view(torch.uint8)[where, :, row] = y
        s[name + "_scale"].copy_(new.unflatten(0, (-1, blocks)).transpose(1, 2))


def _rows_of(s, name):
    """The cached rows of every request, [bs, Hkv, positions, 128] in 32 bits."""
    c, pt = s["case"], s["page_table"].long()
    x = s[name + "_cache"].view(torch.uint8)[pt].view(torch.float8_e4m3fn).float()
    x = x * s[name + "_scale"][pt].repeat_interleave(c["block"], -1)[..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attn(s):
    c = s["case"]
    dev = s["q"].device
    cu = s["cu_seqlens_q"].long()
    count, first = cu[1:] - cu[:-1], cu[:-1]
    node = torch.arange(s["max_q_len"], device=dev)
    row = (first[:, None] + node).clamp(max=s["q"].shape[0] - 1)
    group = c["hq"] // c["hkv"]
    q = s["q"][row].float().unflatten(2, (c["hkv"], group)).transpose(1, 2).flatten(2, 3)
    x = q @ _rows_of(s, "k").transpose(2, 3) * SM_SCALE
    last = s["cache_seqlens"].long()[:, None] - count[:, None] + node  # a query's own position
    seen = torch.arange(x.shape[-1], device=dev) <= last.repeat_interleave(group, 1)[..., None]
    x = x.masked_fill(~seen[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = (p @ _rows_of(s, "v")) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total)).squeeze(-1)
    live = node < count[:, None]

    def back(y):  # [bs, Hkv, new * G, ...] -> [rows, Hq, ...]
        y = y.unflatten(2, (s["max_q_len"], group)).transpose(1, 2).flatten(2, 3)
        return y[live]

    s["out"].copy_(back(o))
    s["lse"].copy_(back(lse))


def _plain_verify(s):
    c = s["case"]
    bs, new, vocab = c["bs"], c["new"], c["vocab"]
    dev = s["tokens"].device
    p, u = s["target_probs"], s["uniforms"].double().view(bs, new)
    tokens = s["tokens"].view(bs, new)
    node = torch.arange(new, device=dev)
    base = torch.arange(bs, device=dev)[:, None] * new
    drafted = node > 0
    if c["tree"]:
        parents = s["parents"].long().view(bs, new)
        pv = p[base + parents.clamp(min=0), tokens].double()
        # siblings before a node (of those with one token, the first counts)
        before = (parents[:, :, None] == parents[:, None]) & (node[:, None] > node) & drafted
        same = before & (tokens[:, :, None] == tokens[:, None])
        first = ~same.any(-1)
        left = 1.0 - (before & first[:, None]).double().mul(pv[:, None]).sum(-1)
        fits = drafted & first & (u * left < pv)
        chosen = fits & ~(before & fits[:, None]).any(-1)
        chosen[:, 0] = True
        bits = (chosen.long() << node).sum(-1, keepdim=True)
        path = (s["masks"] & ~bits) == 0
    else:
        up = base + (node - 1).clamp(min=0)
        ok = u * s["draft_probs"][up, tokens].double() < p[up, tokens].double()
        path = torch.cumprod((ok | ~drafted).int(), -1).bool()
    last = torch.where(path, node, 0).amax(-1)
    w = p[base[:, 0] + last].double()
    if c["tree"]:
        gone = (parents == last[:, None]) & drafted
        w = w.scatter_reduce(1, tokens, torch.where(gone, 0.0, math.inf).double(), "amin")
    elif new > 1:
        q = s["draft_probs"][base[:, 0] + last].double()
        w = torch.where(last[:, None] < new - 1, (w - q).float().double().clamp(min=0), w)
    total = torch.cumsum((w.clamp(max=1) * UNITS).long(), -1)
    t = torch.floor(s["final_uniforms"].double() * total[:, -1].double()).long()
    s["next_tokens"].copy_((total <= t[:, None]).sum(-1))
    begin = s["cache_seqlens"].long() - new
    order = torch.argsort(~path, dim=-1, stable=True)
    count = path.sum(-1)
    s["kept"].copy_(torch.where(node < count[:, None], begin[:, None] + order, -1))
    s["counts"].copy_(count)
    s["begin"].copy_(begin)


def _plain_fork(s):
    page = s["case"]["page"]
    table, refs, n = s["req_to_token"], s["page_refs"], s["lens"].long()
    width = s["max_seq_pages"]
    col = torch.arange(width, device=n.device)
    # the children of the pass before: their pages given back
    first = table[s["children"]][:, ::page]
    given = (col < -(-n // page)[:, None]) & (first >= 0)
    refs.index_add_(0, torch.where(given, first // page, 0).flatten().long(),
                    -given.flatten().int())
    mine = table[s["children"]].unflatten(1, (width, page))
    mine[..., 0] = torch.where(given, -1, mine[..., 0])
    # the forks: full pages shared, the last page copied to the lowest free one
    full = n // page
    partial = n % page > 0
    free = torch.argsort((refs != 0).int(), stable=True)
    fresh = free[(torch.cumsum(partial, 0) - 1).clamp(min=0)]
    theirs = table[s["parents"]].unflatten(1, (width, page))
    slots = fresh[:, None] * page + torch.arange(page, device=n.device)
    mine = torch.where((col < full[:, None])[..., None], theirs, mine)
    here = (col == full[:, None]) & partial[:, None]
    mine = torch.where(here[..., None], slots[:, None].int(), mine)
    table[s["children"]] = mine.flatten(1)
    shared = col < full[:, None]
    refs.index_add_(0, torch.where(shared, theirs[..., 0] // page, 0).flatten().long(),
                    shared.flatten().int())
    took = torch.nonzero(partial)[:, 0]
    refs[fresh[took]] = 1
    src = theirs[took, full[took], 0].long() // page
    for pool in s["pools"]:
        pool = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        pool[fresh[took]] = pool[src]
    s["child_lens"].copy_(n)


def _plain_compact(s):
    page = s["case"]["page"]
    table, refs = s["req_to_token"], s["page_refs"]
    table.copy_(s["scattered"][0])
    refs.copy_(s["scattered"][1])
    live = refs > 0
    index = torch.arange(refs.shape[0], device=refs.device)
    count = live.sum()
    src = torch.nonzero(live & (index >= count))[:, 0]
    dst = torch.nonzero(~live & (index < count))[:, 0]
    s["page_map"].copy_(torch.where(live, index, -1))
    s["page_map"][src] = dst.int()
    refs[dst] = refs[src]
    refs[src] = 0
    s["num_live"].copy_(count)
    for pool in s["pools"]:
        pool = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        pool[dst] = pool[src]
    width = s["max_seq_pages"]
    mine = table[s["rows"]].unflatten(1, (width, page))
    held = torch.arange(width, device=refs.device) < -(-s["lens"].long() // page)[:, None]
    to = s["page_map"][torch.where(held, mine[..., 0] // page, 0).long()]
    slots = to[..., None] * page + torch.arange(page, device=refs.device)
    table[s["rows"]] = torch.where(held[..., None], slots.int(), mine).flatten(1)


# ---- the library's calls ----------------------------------------------------------------------


def _prepared(s):
    """The library's calls on the state's buffers, marshalled once like a serving loop's."""
    from paged_kv_decode_metadata_gb300 import binding as B

    c = s["case"]
    if c["op"] == "append":
        return [B.prepare_rope_append_blocks(
            q=s["q"], k=s["k"], v=s["v"], positions=s["positions"], inv_freq=s["inv_freq"],
            interleaved=c["interleaved"], q_out=s["q_out"], cu_seqlens_q=s["cu_seqlens_q"],
            cache_seqlens=s["cache_seqlens"], page_table=s["page_table"],
            max_seq_pages=s["max_seq_pages"], k_cache=s["k_cache"],
            v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])]
    if c["op"] == "attn":
        size = B.pa_block_workspace_bytes(c["bs"], s["q"].shape[0], s["max_q_len"], c["hq"],
                                          c["hkv"], HEAD_DIM, c["page"], s["max_seq_pages"])
        return [B.prepare_block_attention(
            q=s["q"], k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"],
            v_scale=s["v_scale"], page_table=s["page_table"], cache_seqlens=s["cache_seqlens"],
            cu_seqlens_q=s["cu_seqlens_q"], max_q_len=s["max_q_len"],
            max_seq_pages=s["max_seq_pages"], num_splits=0, sm_scale=SM_SCALE,
            workspace=torch.empty(size, dtype=torch.uint8, device="cuda"), out=s["out"],
            lse=s["lse"])]
    if c["op"] == "verify":
        return [B.prepare_verify_drafts(
            target_probs=s["target_probs"], draft_probs=s["draft_probs"], tokens=s["tokens"],
            parents=s["parents"], cu_seqlens_q=s["cu_seqlens_q"],
            cache_seqlens=s["cache_seqlens"], uniforms=s["uniforms"],
            final_uniforms=s["final_uniforms"], max_q_len=c["new"], kept=s["kept"],
            counts=s["counts"], begin=s["begin"], next_tokens=s["next_tokens"])]
    common = dict(req_to_token=s["req_to_token"], page_refs=s["page_refs"], page_size=c["page"],
                  max_seq_pages=s["max_seq_pages"], lens=s["lens"])
    size = B.pa_pages_workspace_bytes(s["page_refs"].numel(), s["lens"].numel())
    workspace = torch.empty(size, dtype=torch.uint8, device="cuda")
    if c["op"] == "fork":
        return [B.prepare_pages_free(rows=s["children"], **common),
                B.prepare_pages_fork(parents=s["parents"], children=s["children"],
                                     pools=s["pools"], child_lens=s["child_lens"],
                                     workspace=workspace, **common)]
    return [B.prepare_pages_compact(rows=s["rows"], pools=s["pools"], page_map=s["page_map"],
                                    num_live=s["num_live"], workspace=workspace, **common)]


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if own:
        if "calls" not in s:
            s["calls"] = _prepared(s)
        if op == "compact":  # the scattered state put back
            s["req_to_token"].copy_(s["scattered"][0])
            s["page_refs"].copy_(s["scattered"][1])
        for call in s["calls"]:
            call()
    else:
        {"append": _plain_append, "attn": _plain_attn, "verify": _plain_verify,
         "fork": _plain_fork, "compact": _plain_compact}[op](s)
    if op == "attn":
        return {"out": s["out"], "lse": s["lse"]}
    if op == "verify":
        return {x: s[x] for x in ("kept", "counts", "begin", "next_tokens")}
    if op == "append":  # (an e4m3 tensor has the codes' values, a block's scale is beside it)
        return {x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale", "q_out")}
    got = {"pools": s["pools"], "table": s["req_to_token"], "refs": s["page_refs"]}
    return got | {x: s[x] for x in (("child_lens",) if op == "fork" else ("page_map", "num_live"))}


# ---- the definitions in 64 bits ---------------------------------------------------------------


def _to_code(x):
    """The nearest e4m3 value (ties to even) of finite 64-bit values, saturated."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-CODE_MAX, CODE_MAX)


def exact(case, seed):
    c = case
    if c["op"] not in ("append", "attn"):
        return None  # tokens are chosen and pages moved, no values are computed
    s = prepare(case, seed)
    n, d = lengths(c), _new(c)
    page, block = c["page"], c["block"]
    group = c["hq"] // c["hkv"]

    def request(b, name):
        """Positions of request b, [n, Hkv, 128] in 64 bits."""
        j = torch.arange(n[b], device="cuda")
        p = s["page_table"][b].long()[j // page]
        x = s[name + "_cache"].view(torch.uint8)[p, :, j % page].view(torch.float8_e4m3fn)
        return x.double() * s[name + "_scale"][p, :, j % page // block].double()[..., None]

    if c["op"] == "attn":
        out, lse = s["out"].double(), s["lse"].double()
        at = 0
        for b in range(c["bs"]):
            k, v = request(b, "k"), request(b, "v")
            own_at = n[b] - d[b] + torch.arange(d[b], device="cuda").repeat_interleave(group)
            hidden = torch.arange(n[b], device="cuda") > own_at[:, None]
            for h in range(c["hkv"]):
                heads = slice(h * group, (h + 1) * group)
                q = s["q"][at:at + d[b], heads].double().reshape(-1, HEAD_DIM)
                x = ((q @ k[:, h].T) * SM_SCALE).masked_fill(hidden, -math.inf)
                total = torch.logsumexp(x, -1, keepdim=True)
                o = torch.exp(x - total) @ v[:, h]
                out[at:at + d[b], heads] = o.view(d[b], group, HEAD_DIM)
                lse[at:at + d[b], heads] = total.view(d[b], group)
            at += d[b]
        return {"out": out, "lse": lse}

    z = torch.polar(torch.ones_like(s["inv_freq"])[None],
                    s["positions"].double()[:, None] * s["inv_freq"])[:, None]

    def turn(x):
        y = x.double().clone()
        half = c["rot"] // 2
        i = torch.arange(half, device=y.device)
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        w = torch.complex(y[..., a], y[..., b]) * z
        y[..., a], y[..., b] = w.real, w.imag
        return y

    got = {"q_out": turn(s["q"])}
    for name, x in (("k", turn(s["k"])), ("v", s["v"].double())):
        scale = s[name + "_scale"].double()
        codes = s[name + "_cache"].double().unflatten(2, (-1, block))
        at = 0
        for b in range(c["bs"]):
            if d[b] > block and b > 3:  # (a block at a time: it would take too long)
                return None
            for k in range((n[b] - d[b]) // block, (n[b] - 1) // block + 1):
                lo, hi = max(k * block, n[b] - d[b]), min((k + 1) * block, n[b])
                rows = x[at + lo - n[b] + d[b]:at + hi - n[b] + d[b]].transpose(0, 1)
                p = int(s["page_table"][b, lo // page])
                i, r = k % (page // block), lo - k * block
                want = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((1, 2)) / CODE_MAX)))
                old = scale[p, :, i].clone()
                new = torch.maximum(old, want) if r else want
                codes[p, :, i, :r] = _to_code(codes[p, :, i, :r] * (old / new)[:, None, None])
                codes[p, :, i, r:r + hi - lo] = _to_code(rows / new[:, None, None])
                scale[p, :, i] = new
            at += d[b]
        got |= {name + "_cache": codes.flatten(2, 3), name + "_scale": scale}
    return got
