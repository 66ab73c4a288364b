"""Cases of the cache operators, in plain PyTorch and through the library.

Four operators of a decode loop over the paged K/V pools ([num_pages, Hkv, page_size, 128],
bf16, or int8 codes with an fp32 scale per row):

* ``rope``     rotary positions applied to the new queries and keys, and the new keys and
               values written to their slots of the pools (quantised for int8 pools);
* ``tree``     attention of the drafted tokens of a speculation tree over the cache: every
               committed position, and the node's own ancestors;
* ``weights``  the decode step's attention weights added up per cached row;
* ``evict``    the rows with the largest accumulated weights kept, with the first and the
               newest ones, and moved in order to the request's new pages.

``listed`` holds the cases, ``draw`` more of the same ranges, ``run`` one pass: through
elementary torch operations in 32 bits, or, where ``own`` is set, through the library.
"""

import math
import random

import torch

own = False

HEAD_DIM = 128
SM_SCALE = float(torch.tensor(HEAD_DIM ** -0.5, dtype=torch.float32))
ROPE_BASE = 10000.0


def listed():
    return [
        # one new token for each of 32 decoding requests: launch latency counts
        dict(name="rope_decode_32", op="rope", tokens=32, hq=32, hkv=8, page=64, kv="bf16",
             rot=128, interleaved=False, scaling="none", start=8000, padded=0, decode=True),
        # a prompt chunk entering the cache
        dict(name="rope_prompt_8k", op="rope", tokens=8192, hq=32, hkv=8, page=64, kv="bf16",
             rot=128, interleaved=False, scaling="none", start=0, padded=0, decode=False),
        # a ragged chunk far into a long context: half of the head rotates, frequencies
        # interpolated by parts, int8 pool, some rows padding
        dict(name="rope_int8_far_4097", op="rope", tokens=4097, hq=64, hkv=8, page=64, kv="int8",
             rot=64, interleaved=True, scaling="by_parts", start=500000, padded=100,
             decode=False),
        # one request verifying a small draft
        dict(name="tree_bs1_1k", op="tree", bs=1, ctx=1024, ragged=False, nodes=8, hq=32, hkv=8,
             page=64, kv="bf16"),
        # a small ragged batch, no shared heads, small pages, odd lengths and drafts
        dict(name="tree_bs8_ragged", op="tree", bs=8, ctx=4001, ragged=True, nodes=23, hq=16,
             hkv=16, page=16, kv="bf16"),
        # the serving batch: 32 requests at 8K tokens, 32 drafted tokens each
        dict(name="tree_bs32_8k", op="tree", bs=32, ctx=8192, ragged=False, nodes=32, hq=32, hkv=8,
             page=64, kv="bf16"),
        # the ragged int8 batch up to 16K tokens
        dict(name="tree_bs64_ragged_int8", op="tree", bs=64, ctx=16384, ragged=True, nodes=32,
             hq=64, hkv=8, page=64, kv="int8"),
        # large trees over long contexts: the products, not the cache, set the time
        dict(name="tree_bs16_16k_64", op="tree", bs=16, ctx=16384, ragged=False, nodes=64, hq=64,
             hkv=8, page=128, kv="bf16"),
        # accumulated weights of one long request
        dict(name="weights_bs1_8k", op="weights", bs=1, ctx=8192, ragged=False, hq=32, hkv=8,
             page=64, kv="bf16"),
        # ... and of the ragged int8 batch
        dict(name="weights_bs64_ragged_int8", op="weights", bs=64, ctx=16384, ragged=True, hq=64,
             hkv=8, page=64, kv="int8"),
        # one request shrunk to an eighth
        dict(name="evict_bs1_8k", op="evict", bs=1, ctx=8192, ragged=False, hq=8, hkv=8, page=64,
             kv="bf16", budget=1024, first=4, recent=256),
        # a batch shrunk to a quarter at once (memory pressure)
        dict(name="evict_bs32_8k", op="evict", bs=32, ctx=8192, ragged=False, hq=8, hkv=8, page=64,
             kv="bf16", budget=2048, first=4, recent=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "tree", "tree", "weights", "evict"])
        hkv = rng.choice([1, 2, 4, 8, 16])
        hq = hkv * rng.choice([1, 2, 4, 8, 16])
        c = dict(op=op, hq=hq, hkv=hkv, page=rng.choice([16, 32, 64, 128]),
                 kv=rng.choice(["bf16", "int8"]))
        if op == "rope":
            tokens = _log_int(rng, 1, 8192)
            c.update(tokens=tokens, rot=16 * rng.randint(1, 8), interleaved=rng.random() < 0.5,
                     scaling=rng.choice(["none", "by_parts"]), start=_log_int(rng, 1, 1000000),
                     padded=rng.randint(0, tokens // 8),
                     decode=tokens <= 256 and rng.random() < 0.5)
        else:
            c.update(bs=_log_int(rng, 1, 64), ctx=_log_int(rng, 64, 16384),
                     ragged=rng.random() < 0.5)
            if op == "tree":
                c.update(nodes=rng.randint(1, 64))
            if op == "evict":
                budget = _log_int(rng, 16, max(17, c["ctx"] // 2))
                recent = rng.randint(0, budget // 2)
                c.update(budget=budget, first=min(4, budget - recent), recent=recent)
        w = work(c)
        # no more than the largest listed case of bytes and of products
        if w["bytes"] <= 1.1e9 and w["flops"] <= 5.0e11:
            return c


# ---- lengths: fixed by the case, so that its work does not depend on the seed -----------


def lengths(c):
    """Cached tokens of each request (drafted ones among them)."""
    if not c["ragged"]:
        return [c["ctx"]] * c["bs"]
    n = [max(1, (2 * i + 1) * c["ctx"] // (2 * c["bs"])) for i in range(c["bs"])]
    random.Random(c["bs"] * 100003 + c["ctx"]).shuffle(n)
    return n


def draft_lengths(c):
    """Drafted tokens of each request: up to ``nodes``, no more than it has cached."""
    r = random.Random(c["bs"] * 7919 + c["nodes"])
    want = [r.randint(1, c["nodes"]) if c["ragged"] else c["nodes"] for _ in range(c["bs"])]
    return [min(a, b) for a, b in zip(want, lengths(c))]


def _row_bytes(c):
    return HEAD_DIM * 2 if c["kv"] == "bf16" else HEAD_DIM + 4


def work(c):
    row = _row_bytes(c)
    if c["op"] == "rope":
        rows = c["tokens"] * (c["hq"] + 2 * c["hkv"])
        stored = (c["tokens"] - c["padded"]) * 2 * c["hkv"]
        flops = 6 * c["tokens"] * (c["hq"] + c["hkv"]) * c["rot"] // 2
        return {"bytes": rows * 256 + c["tokens"] * (c["hq"] * 256 + 16) + stored * row,
                "flops": flops}
    n = lengths(c)
    kv = sum(n) * c["hkv"] * row
    if c["op"] == "tree":
        d = draft_lengths(c)
        rows = sum(d) * c["hq"]
        pairs = sum(di * (ni - di + 1) for di, ni in zip(d, n)) * c["hq"]
        return {"bytes": 2 * kv + rows * (512 + 4) + sum(d) * 8, "flops": 4 * HEAD_DIM * pairs}
    if c["op"] == "weights":
        return {"bytes": kv + sum(n) * c["hkv"] * 8 + c["bs"] * c["hq"] * 260,
                "flops": 2 * HEAD_DIM * sum(n) * c["hq"]}
    kept = sum(min(x, c["budget"]) for x in n) * c["hkv"]
    return {"bytes": 2 * kept * (2 * row + 4) + kept * 4 + sum(n) * c["hkv"] * 4, "flops": sum(n)}


# ---- inputs ---------------------------------------------------------------------------------


def inverse_frequencies(c):
    """Radians per position of each rotated pair, in 64 bits.  ``by_parts``: pairs that turn
    more than 32 times over the original 4096 positions keep their frequency, those that
    turn less than once are slowed 32 times, a linear ramp in between."""
    half = c["rot"] // 2
    i = torch.arange(half, dtype=torch.float64)
    f = ROPE_BASE ** (-2.0 * i / c["rot"])
    if c["scaling"] == "none":
        return f
    where = [c["rot"] * math.log(4096 / (2 * math.pi * t)) / (2 * math.log(ROPE_BASE))
             for t in (32.0, 1.0)]
    lo, hi = max(0, math.floor(where[0])), min(c["rot"] - 1, math.ceil(where[1]))
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f / 32.0 * ramp + f * (1 - ramp)


def _pool(c, num_pages, g, dev):
    shape = (num_pages, c["hkv"], c["page"], HEAD_DIM)
    if c["kv"] == "bf16":
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16), None
    codes = torch.randint(-127, 128, shape, generator=g, device=dev, dtype=torch.int8)
    return codes, torch.rand(shape[:3], generator=g, device=dev) * 0.045 + 0.005


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": c}

    def trees():
        """Ancestor masks (bit t of node i: node t is i or above it) of seeded trees."""
        r = random.Random(seed)
        rows = []
        for d in draft_lengths(c):
            own_rows = []
            for i in range(d):
                parent = r.randint(max(-1, i - 9), i - 1) if i else -1
                own_rows.append((own_rows[parent] if parent >= 0 else 0) | (1 << i))
            rows += own_rows
        return torch.tensor([m - (1 << 64) if m >> 63 else m for m in rows], dtype=torch.int64)

    if c["op"] == "rope":
        t, heads = c["tokens"], c["hq"] + 2 * c["hkv"]
        # one projection's output: q, k and v are views of its rows
        qkv = torch.randn((t, heads, HEAD_DIM), generator=g, device=dev, dtype=torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        at = torch.arange(t, device=dev)
        if c["decode"]:  # one token of each request, somewhere in its last page
            pages = t + 1
            s["positions"] = torch.randint(c["start"], 2 * c["start"] + 1, (t,), generator=g,
                                           device=dev)
            at = at * c["page"] + s["positions"] % c["page"]
        else:  # consecutive tokens of one request
            pages = -(-t // c["page"]) + 1
            s["positions"] = c["start"] + at
        order = torch.randperm(pages, generator=g, device=dev)
        slots = order[at // c["page"]] * c["page"] + at % c["page"]
        slots[t - c["padded"]:] = -1
        s["slots"] = slots
        s["inv_freq"] = inverse_frequencies(c).to(dev)
        s["amplitude"] = 0.1 * math.log(32.0) + 1.0 if c["scaling"] == "by_parts" else 1.0
        s["k_cache"], s["k_scale"] = _pool(c, pages, g, dev)
        s["v_cache"], s["v_scale"] = _pool(c, pages, g, dev)
        s["q_out"] = torch.empty((t, c["hq"], HEAD_DIM), dtype=torch.bfloat16, device=dev)
        if c["kv"] == "int8":  # room for the values that codes and scales stand for
            s["values"] = [torch.empty(s["k_cache"].shape, dtype=torch.bfloat16, device=dev)
                           for _ in "kv"]
        return s
    n = lengths(c)
    per = [-(-x // c["page"]) for x in n]
    msp = max(per)
    new = [-(-min(x, c.get("budget", 0)) // c["page"]) for x in n]
    total = sum(per) + sum(new)
    order = torch.randperm(total, generator=g, device=dev, dtype=torch.int32)
    lens = torch.tensor(n, device=dev, dtype=torch.int32)
    s["cache_seqlens"] = lens

    def table(counts, begin, width):
        count = torch.tensor(counts, device=dev)
        first = begin + torch.cumsum(count, 0) - count
        col = torch.arange(width, device=dev)
        at = (first[:, None] + col).clamp(max=total - 1)
        return torch.where(col < count[:, None], order[at], 0).to(torch.int32).contiguous()

    s["page_table"] = table(per, 0, msp)
    s["max_seq_pages"] = msp
    s["k_cache"], s["k_scale"] = _pool(c, total, g, dev)
    if c["op"] != "weights":
        s["v_cache"], s["v_scale"] = _pool(c, total, g, dev)
    wshape = (total, c["hkv"], c["page"])
    if c["op"] == "evict":
        # heavy-tailed accumulated weights; a tenth of the rows were never attended to
        w = torch.rand(wshape, generator=g, device=dev).pow(8) * 50
        s["weights"] = torch.where(torch.rand(wshape, generator=g, device=dev) < 0.1, 0.0, w)
        s["dst_page_table"] = table(new, sum(per), max(new))
        s["kept"] = torch.empty((c["bs"], c["hkv"], c["budget"]), dtype=torch.int32, device=dev)
        s["new_seqlens"] = torch.empty(c["bs"], dtype=torch.int32, device=dev)
        return s
    if c["op"] == "weights":
        s["q"] = torch.randn((c["bs"], c["hq"], HEAD_DIM), generator=g, device=dev,
                             dtype=torch.bfloat16)
        s["weights"] = torch.rand(wshape, generator=g, device=dev)
        x = _scores(s, s["q"].view(c["bs"], 1, c["hq"], HEAD_DIM))
        seen = torch.arange(x.shape[-1], device=dev) < lens[:, None]
        s["lse"] = torch.logsumexp(x.masked_fill(~seen[:, None, None], -math.inf), -1) \
            .view(c["bs"], c["hq"]).contiguous()
        return s
    d = draft_lengths(c)
    rows = sum(d)
    s["q"] = torch.randn((rows, c["hq"], HEAD_DIM), generator=g, device=dev, dtype=torch.bfloat16)
    s["max_q_len"] = max(d)
    s["cu_seqlens_q"] = torch.tensor([sum(d[:i]) for i in range(len(d) + 1)], device=dev,
                                     dtype=torch.int32)
    s["tree_mask"] = trees().view(rows, 1).to(dev)
    s["out"] = torch.empty((rows, c["hq"], HEAD_DIM), dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.empty((rows, c["hq"]), dtype=torch.float32, device=dev)
    return s


# ---- the plain forms ------------------------------------------------------------------------


def _values(codes, scale):
    """Rows of a pool in 32 bits."""
    return codes.float() if scale is None else codes.float() * scale[..., None]


def _rows_of(s, name):
    """The cached rows of every request, [bs, Hkv, positions, 128] in 32 bits."""
    pt = s["page_table"].long()
    scale = s[name + "_scale"]
    rows = _values(s[name + "_cache"][pt], None if scale is None else scale[pt])
    return rows.transpose(1, 2).flatten(2, 3)


def _scores(s, q):
    """Scaled scores of query rows q [bs, rows, Hq, 128]: [bs, Hkv, rows * G, positions]."""
    bs, rows, hq, _ = q.shape
    hkv = s["case"]["hkv"]
    q = q.float().view(bs, rows, hkv, hq // hkv, HEAD_DIM).transpose(1, 2).flatten(2, 3)
    return q @ _rows_of(s, "k").transpose(2, 3) * SM_SCALE


def _quantised(x):
    """Symmetric int8 rows: codes and scales."""
    scale = x.abs().amax(-1) / 127
    inverse = torch.where(scale > 0, 1 / scale, 0.0)
    return torch.round(x * inverse[..., None]).clamp(-127, 127).to(torch.int8), scale


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos = (torch.cos(angle) * s["amplitude"]).float()[:, None]
    sin = (torch.sin(angle) * s["amplitude"]).float()[:, None]

    def rotated(x):
        x = x.float()
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else r.chunk(2, -1)
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((r, rest), -1)

    s["q_out"].copy_(rotated(s["q"]))
    live = s["slots"] >= 0
    slots = s["slots"][live]
    page, row = slots // c["page"], slots % c["page"]
    k, v = rotated(s["k"])[live], s["v"].float()[live]
    if c["kv"] == "int8":
        k, s["k_scale"][page, :, row] = _quantised(k)
        v, s["v_scale"][page, :, row] = _quantised(v)
    s["k_cache"][page, :, row] = k.to(s["k_cache"].dtype)
    s["v_cache"][page, :, row] = v.to(s["v_cache"].dtype)


def _plain_tree(s):
    c = s["case"]
    dev = s["q"].device
    cu = s["cu_seqlens_q"].long()
    count, first = cu[1:] - cu[:-1], cu[:-1]
    node = torch.arange(s["max_q_len"], device=dev)
    row = (first[:, None] + node).clamp(max=s["q"].shape[0] - 1)
    x = _scores(s, s["q"][row])
    pos = torch.arange(x.shape[-1], device=dev)
    n = s["cache_seqlens"].long()
    t = pos - (n - count)[:, None]
    bit = (s["tree_mask"][row, 0][..., None] >> t.clamp(0, 63)[:, None]) & 1
    seen = (t < 0)[:, None] | ((t >= 0) & (t < count[:, None]))[:, None] & (bit == 1)
    group = c["hq"] // c["hkv"]
    seen = seen.repeat_interleave(group, 1)[:, None]
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = (p @ _rows_of(s, "v")) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total)).squeeze(-1)
    live = node < count[:, None]

    def back(y):  # [bs, Hkv, nodes * G, ...] -> [rows, Hq, ...]
        y = y.unflatten(2, (s["max_q_len"], group)).transpose(1, 2).flatten(2, 3)
        return y[live]

    s["out"].copy_(back(o))
    s["lse"].copy_(back(lse))


def _plain_weights(s):
    c = s["case"]
    x = _scores(s, s["q"].view(c["bs"], 1, c["hq"], HEAD_DIM))
    pos = torch.arange(x.shape[-1], device=x.device)
    seen = pos < s["cache_seqlens"][:, None]
    p = torch.exp(x - s["lse"].view(c["bs"], c["hkv"], -1, 1)).sum(2)
    p = torch.where(seen[:, None], p, 0.0).unflatten(2, (-1, c["page"])).transpose(1, 2)
    s["weights"].index_add_(0, s["page_table"].flatten(), p.flatten(0, 1))


def _plain_evict(s):
    c = s["case"]
    dev = s["weights"].device
    n = s["cache_seqlens"].long()[:, None, None]
    w = s["weights"][s["page_table"].long()].transpose(1, 2).flatten(2, 3)
    pos = torch.arange(w.shape[-1], device=dev)
    always = (pos < c["first"]) | (pos >= n - c["recent"])
    w = torch.where(always, math.inf, w)
    w = torch.where(pos < n, w, -math.inf)
    budget = min(c["budget"], w.shape[-1])
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    rank = torch.arange(budget, device=dev)
    order = torch.where(rank < n, order, w.shape[-1])  # a request shorter than the budget
    order = torch.sort(order, dim=-1).values
    s["kept"].fill_(-1)
    s["kept"][..., :budget] = torch.where(rank < n, order, -1)
    s["new_seqlens"].copy_(n.flatten().clamp(max=c["budget"]))
    b, h, i = torch.nonzero(s["kept"] >= 0, as_tuple=True)
    j = s["kept"][b, h, i].long()
    src = (s["page_table"].long()[b, j // c["page"]], h, j % c["page"])
    dst = (s["dst_page_table"].long()[b, i // c["page"]], h, i % c["page"])
    s["weights"][dst] = s["weights"][src]
    s["k_cache"][dst] = s["k_cache"][src]
    s["v_cache"][dst] = s["v_cache"][src]
    if c["kv"] == "int8":
        s["k_scale"][dst] = s["k_scale"][src]
        s["v_scale"][dst] = s["v_scale"][src]


# ---- the library's calls ----------------------------------------------------------------------


def _prepared(s):
    """The library's call on the state's buffers, marshalled once like a serving loop's."""
    from paged_kv_decode_metadata_gb300 import binding as B

    c = s["case"]
    if c["op"] == "rope":
        return B.prepare_rope_append(
            q=s["q"], k=s["k"], v=s["v"], positions=s["positions"], slots=s["slots"],
            inv_freq=s["inv_freq"], interleaved=c["interleaved"], amplitude=s["amplitude"],
            q_out=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"],
            v_scale=s["v_scale"])
    if c["op"] == "tree":
        size = B.pa_tree_workspace_bytes(c["bs"], s["q"].shape[0], s["max_q_len"], c["hq"],
                                         c["hkv"], HEAD_DIM, c["page"], s["max_seq_pages"])
        return B.prepare_tree_attention(
            q=s["q"], k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"],
            v_scale=s["v_scale"], page_table=s["page_table"], cache_seqlens=s["cache_seqlens"],
            cu_seqlens_q=s["cu_seqlens_q"], tree_mask=s["tree_mask"], max_q_len=s["max_q_len"],
            max_seq_pages=s["max_seq_pages"], num_splits=0, sm_scale=SM_SCALE,
            workspace=torch.empty(size, dtype=torch.uint8, device="cuda"), out=s["out"],
            lse=s["lse"])
    if c["op"] == "weights":
        return B.prepare_accumulate_weights(
            q=s["q"], lse=s["lse"], k_cache=s["k_cache"], k_scale=s["k_scale"],
            page_table=s["page_table"], cache_seqlens=s["cache_seqlens"], weights=s["weights"],
            max_seq_pages=s["max_seq_pages"], sm_scale=SM_SCALE)
    return B.prepare_evict(
        page_table=s["page_table"], cache_seqlens=s["cache_seqlens"], weights=s["weights"],
        k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"],
        max_seq_pages=s["max_seq_pages"], budget=c["budget"], num_first=c["first"],
        num_recent=c["recent"], dst_page_table=s["dst_page_table"], kept=s["kept"],
        new_seqlens=s["new_seqlens"])


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        if "call" not in s:
            s["call"] = _prepared(s)
        s["call"]()
    else:
        {"rope": _plain_rope, "tree": _plain_tree, "weights": _plain_weights,
         "evict": _plain_evict}[op](s)
    if op == "tree":
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weights":
        return {"weights": s["weights"]}
    got = {"k": s["k_cache"], "v": s["v_cache"]}
    if s["case"]["kv"] == "int8":
        if op == "rope":
            got = {x: torch.mul(s[x + "_cache"], s[x + "_scale"][..., None], out=y)
                   for x, y in zip("kv", s["values"])}
        got |= {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if op == "rope":
        return got | {"q": s["q_out"]}
    return got | {"kept": s["kept"], "new_seqlens": s["new_seqlens"], "weights": s["weights"]}


# ---- the definitions in 64 bits ---------------------------------------------------------------


def exact(case, seed):
    if case["op"] == "evict":
        return None  # rows are moved, nothing is computed
    c, s = case, prepare(case, seed)

    def exact_rope():
        z = torch.polar(torch.full_like(s["inv_freq"], s["amplitude"])[None],
                        s["positions"].double()[:, None] * s["inv_freq"])[:, None]

        def turn(x):
            y = x.double().clone()
            half = c["rot"] // 2
            i = torch.arange(half, device=y.device)
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
            w = torch.complex(y[..., a], y[..., b]) * z
            y[..., a], y[..., b] = w.real, w.imag
            return y

        got = {"q": turn(s["q"])}
        for name, x in (("k", turn(s["k"])), ("v", s["v"].double())):
            cache, scale = s[name + "_cache"].double(), s[name + "_scale"]
            if scale is not None:
                scale = scale.double()
            for lo in range(0, c["tokens"] - c["padded"], 1024):
                slot = s["slots"][lo:min(lo + 1024, c["tokens"] - c["padded"])]
                rows = x[lo:lo + slot.shape[0]]
                where = (slot // c["page"], slice(None), slot % c["page"])
                if scale is not None:
                    scale[where] = rows.abs().amax(-1) / 127
                    rows = torch.round(rows / scale[where][..., None])
                cache[where] = rows
            got[name] = cache if scale is None else cache * scale[..., None]
            if scale is not None:
                got[name + "_scale"] = scale
        return got

    def request(b, name):
        """Positions of request b, [n, Hkv, 128] in 64 bits."""
        n, page = int(s["cache_seqlens"][b]), c["page"]
        j = torch.arange(n, device="cuda")
        p = s["page_table"][b].long()[j // page]
        x = s[name + "_cache"][p, :, j % page].double()
        scale = s[name + "_scale"]
        return x if scale is None else x * scale[p, :, j % page].double()[..., None]

    def exact_tree():
        group = c["hq"] // c["hkv"]
        out, lse = s["out"].double(), s["lse"].double()
        at = 0
        for b, d in enumerate(draft_lengths(c)):
            k, v = request(b, "k"), request(b, "v")
            n = k.shape[0]
            masks = s["tree_mask"][at:at + d, 0].tolist()
            hidden = torch.tensor([[not (m >> t) & 1 for t in range(d)] for m in masks],
                                  device="cuda").repeat_interleave(group, 0)
            for h in range(c["hkv"]):
                q = s["q"][at:at + d, h * group:(h + 1) * group].double().reshape(d * group, HEAD_DIM)
                x = (q @ k[:, h].T) * SM_SCALE
                x[:, n - d:][hidden] = -math.inf
                total = torch.logsumexp(x, -1, keepdim=True)
                o = torch.exp(x - total) @ v[:, h]
                out[at:at + d, h * group:(h + 1) * group] = o.view(d, group, HEAD_DIM)
                lse[at:at + d, h * group:(h + 1) * group] = total.view(d, group)
            at += d
        return {"out": out, "lse": lse}

    def exact_weights():
        group = c["hq"] // c["hkv"]
        w = s["weights"].double()
        for b in range(c["bs"]):
            k = request(b, "k")
            j = torch.arange(k.shape[0], device="cuda")
            q = s["q"][b].double().view(c["hkv"], group, HEAD_DIM)
            x = torch.einsum("hgd,nhd->nhg", q, k) * SM_SCALE
            add = torch.exp(x - s["lse"][b].double().view(c["hkv"], group)).sum(-1)
            w[s["page_table"][b].long()[j // c["page"]], :, j % c["page"]] += add
        return {"weights": w}

    return {"rope": exact_rope, "tree": exact_tree, "weights": exact_weights}[c["op"]]()
