"""What the header promises of the cache operators at the edges of a serving loop, beside the
plain cases of test_gpu_cache_ops.py."""

import math
import random

import pytest
import torch

import cache_reference as R
from paged_kv_decode_metadata_gb300 import binding as B
from paged_kv_decode_metadata_gb300 import build
from test_gpu_cache_ops import SCALE, Cache, Tree, evict, random_parents, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    B.load()
    B.pa_read_error_flags(reset=True)
    yield
    assert B.pa_read_error_flags(reset=True) == 0


# ---- accumulated weights of reused rows -----------------------------------------------------


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("hkv,page", [(1, 16), (3, 64)])
def test_append_clears_the_weights_of_the_rows_it_writes(kv, hkv, page):
    """Those rows' weights become 0 in every head; padded tokens' rows, and all others, keep theirs."""
    tokens = 70
    c = Cache([tokens], hkv, page, kv, 5, poison=False)
    x = torch.randn((tokens, 4 * hkv, 128), generator=c.g).to(torch.bfloat16).cuda()
    q, k, v = x.split([2 * hkv, hkv, hkv], dim=1)
    at = torch.randperm(tokens, generator=c.g)
    slots = c.table[0].long()[at // page] * page + at % page
    slots[3], slots[69] = -1, -5
    kw = dict(q=q, k=k, v=v, positions=at.cuda(), slots=slots.cuda(), inv_freq=B.pa_rope_frequencies(128).cuda(),
              q_out=torch.empty((tokens, 2 * hkv, 128), dtype=torch.bfloat16, device="cuda"), k_cache=c.d_k,
              v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs)
    B.pa_rope_append(**kw)                               # without the weights: none change
    assert same_bits(c.d_w, c.weights)
    plain = [t.clone() for t in (kw["q_out"], c.d_k, c.d_v)]
    B.prepare_rope_append(weights=c.d_w, **kw)()
    want = c.weights.clone()
    for s in slots.tolist():
        if s >= 0:
            want[s // page, :, s % page] = 0
    assert same_bits(c.d_w, want)
    for a, b in zip(plain, (kw["q_out"], c.d_k, c.d_v)):
        assert same_bits(a, b)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_loop_adds_up_weights_by_token(kv):
    """Append, verify, keep the path, append, decode, accumulate, evict in place, three times.  The
    host keeps every token's total itself (0 when it is appended); the pool's weight of each
    live row stays that token's, whatever stood in the row before."""
    hq, hkv, page, msp = 8, 2, 16, 24
    n = [200, 37]
    g = torch.Generator().manual_seed(81)
    r = random.Random(82)
    c = Cache([msp * page] * 2, hkv, page, kv, 83, poison=False)
    # rows past the prompt hold what other requests left
    total = c.weights.double()
    for b in range(2):
        j = torch.arange(n[b])
        total[c.table[b].long()[j // page], :, j % page] = 0
    c.d_w.copy_(total.float())
    slack = torch.zeros_like(total)
    freq = B.pa_rope_frequencies(64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()

    def append(count):
        t = sum(count)
        x = torch.randn((t, hq + 2 * hkv, 128), generator=g).to(torch.bfloat16).cuda()
        q, k, v = x.split([hq, hkv, hkv], dim=1)
        where = [(b, n[b] + i) for b in range(2) for i in range(count[b])]
        slots = torch.tensor([int(c.table[b, j // page]) * page + j % page for b, j in where])
        q_out = torch.empty((t, hq, 128), dtype=torch.bfloat16, device="cuda")
        B.pa_rope_append(q=q, k=k, v=v, positions=torch.tensor([j for _, j in where]).cuda(),
                         slots=slots.cuda(), inv_freq=freq.cuda(), q_out=q_out, k_cache=c.d_k, v_cache=c.d_v,
                         k_scale=c.d_ks, v_scale=c.d_vs, weights=c.d_w)
        for b, j in where:                               # a new token has been attended to by none
            at = int(c.table[b, j // page]), slice(None), j % page
            total[at] = slack[at] = 0
        for b in range(2):
            n[b] += count[b]
        c.n, c.d_n = list(n), i32(n)
        return q_out

    def attend(q, count, masks):
        t = Tree(c, count, hq, 0, masks=masks)
        t.q = q.cpu()
        return t.run(0)[1]

    for _ in range(3):
        count = [7, 5]
        parents = [random_parents(r, k) for k in count]
        attend(append(count), count, [m for p in parents for m in R.ancestor_rows(p)])
        begin = [a - b for a, b in zip(n, count)]
        kept = torch.full((2, 1, 7), -1, dtype=torch.int32)
        path = []
        for b, p in enumerate(parents):
            node, nodes = len(p) - 1, []
            while node >= 0:
                nodes.append(begin[b] + node)
                node = p[node]
            path.append(nodes[::-1])
            kept[b, 0, :len(nodes)] = torch.tensor(path[b])
        new = torch.empty(2, dtype=torch.int32, device="cuda")
        B.pa_compact_cache(page_table=c.d_table, cache_seqlens=c.d_n, kept=kept.cuda(),
                           counts=i32([len(p) for p in path]), begin=i32(begin), k_cache=c.d_k,
                           v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs, weights=c.d_w,
                           max_seq_pages=msp, new_seqlens=new)
        n[:] = new.tolist()
        total, slack = R.move([total, slack], c.table, c.table, [[p] * hkv for p in path], begin)
        q = append([1, 1])
        lse = attend(q, [1, 1], [1, 1])
        B.pa_accumulate_weights(q=q, lse=lse, k_cache=c.d_k, k_scale=c.d_ks, page_table=c.d_table,
                                cache_seqlens=c.d_n, weights=c.d_w, max_seq_pages=msp, sm_scale=SCALE)
        ks = c.d_ks.cpu() if kv == "int8" else None
        total, more = R.accumulate(total, q.cpu(), lse.cpu(), c.d_k.cpu(), ks, c.table, n, SCALE)
        slack = slack + more
        c.weights = c.d_w.cpu()
        lists = []
        for b in range(2):
            j = torch.arange(n[b])
            at = c.table[b].long()[j // page], slice(None), j % page
            err = (c.weights[at].double() - total[at]).abs()
            assert bool((err <= slack[at]).all()), float((err - slack[at]).max())
            lists.append([R.kept_positions(c.weights[at][:, h].tolist(), n[b], 60, 2, 20) for h in range(hkv)])
        got, _, _ = evict(c, 60, 2, 20, True)
        for b in range(2):
            for h in range(hkv):
                assert got[b, h].tolist()[:len(lists[b][h])] == lists[b][h]
        total, slack = R.move([total, slack], c.table, c.table, lists, [0, 0])
        n[:] = [min(x, 60) for x in n]


# ---- query rows that no request covers --------------------------------------------------------


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("splits", [1, 3])
def test_rows_before_the_first_request_are_left(kv, splits):
    c = Cache([900, 260], 2, 64, kv, 7)
    t = Tree(c, [4, 6], 8, 8)
    want = t.run(splits)
    front = 3
    rows = t.total + front
    q = torch.zeros((rows, 8, 128), dtype=torch.bfloat16)
    q[front:] = t.q
    mask = torch.full((rows, 1), -1, dtype=torch.int64)
    mask[front:] = R.mask_tensor(t.masks, 1)
    out, lse = t.run(splits, pad=front, q=q.cuda(), tree_mask=mask.cuda(), cu_seqlens_q=(t.cu + front).cuda())
    assert bool((out[:front] == 7.0).all()) and bool((lse[:front] == 7.0).all())
    assert same_bits(out[front:], want[0]) and same_bits(lse[front:], want[1])


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("bs", [3, 40])
def test_rows_of_a_refused_request_are_left(kv, splits, bs):
    """A request with more rows than max_q_len is reported and not run; its rows stay as they were, and
    the others' are right."""
    n = [300 + 37 * i for i in range(bs)]
    q_lens = [4] * bs
    bad = bs - 2
    q_lens[bad] = 5
    c = Cache(n, 2, 64, kv, 17)
    t = Tree(c, q_lens, 8, 18)
    out, lse = t.run(splits, max_q_len=4)
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_SEQLEN_OUT_OF_RANGE
    lo = sum(q_lens[:bad])
    assert bool((out[lo:lo + 5] == 7.0).all()) and bool((lse[lo:lo + 5] == 7.0).all())
    full = t.run(splits)
    out[lo:lo + 5], lse[lo:lo + 5] = full[0][lo:lo + 5], full[1][lo:lo + 5]
    t.check(out, lse)


# ---- long contexts -------------------------------------------------------------------------------


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("nodes", [1, 160])
def test_tree_sums_of_long_contexts(kv, nodes):
    """Near-equal weights and V of one sign over 2^24 - 5 tokens (every page the same), in as many
    units as fill the device.  The tensor cores truncate each sum of 4 tokens to the accumulator's
    2^-23: pieces of 2^18 tokens are 2^16 such steps at most, 2^-7; then the output's rounding,
    2^-8.  (Whole, the sums read 4 % low: fp32 does not hold an addend 2^-22 of its sum.)"""
    n, bs, hkv = 2 ** 24 - 5, 19 if nodes == 1 else 2, 8
    pages = -(-n // 128)
    value = 0.69921875 if kv == "bf16" else 89.0
    pools = {x + "_cache": torch.full((1, hkv, 128, 128), y, dtype=torch.bfloat16 if kv == "bf16" else torch.int8,
                                      device="cuda") for x, y in (("k", 1), ("v", value))}
    if kv == "int8":
        pools |= {x: torch.ones((1, hkv, 128), device="cuda") for x in ("k_scale", "v_scale")}
    rows = bs * nodes
    out = torch.full((rows, hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, hkv), 7.0, device="cuda")
    words = -(-nodes // 64)
    B.pa_tree_attention(q=torch.zeros((rows, hkv, 128), dtype=torch.bfloat16, device="cuda"),
                        page_table=torch.zeros((bs, pages), dtype=torch.int32, device="cuda"),
                        cache_seqlens=torch.full((bs,), n, dtype=torch.int32, device="cuda"),
                        cu_seqlens_q=torch.arange(bs + 1, dtype=torch.int32, device="cuda") * nodes,
                        tree_mask=torch.full((rows, words), -1, dtype=torch.int64, device="cuda"),
                        max_q_len=nodes, max_seq_pages=pages, sm_scale=SCALE, out=out, lse=lse,
                        workspace=torch.empty(B.pa_tree_workspace_bytes(bs, rows, nodes, hkv, hkv, 128, 128, pages),
                                              dtype=torch.uint8, device="cuda"), **pools)
    torch.cuda.synchronize()
    assert B.pa_read_error_flags(reset=True) == 0
    err = (out.cpu().double() / value - 1).abs().max()
    assert float(err) <= 2.0 ** -7 + 2.0 ** -8, float(err)
    assert float((lse.cpu().double() - math.log(n)).abs().max()) <= 2.0 ** -20 * math.log(n)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_tree_blocks_that_work_for_seconds(kv):
    """2^29 - 1 tokens (a table's most, less one; every page the same) in as many units as fill the
    device: no wait gives up although a block's cut V tile comes seconds after its start.  All
    scores are 0 and V is 1, -1 or 0: the sums of 2^18 tokens, and of 2^11 pieces of them, are
    integers that fp32 holds exactly, but for the last token's of 2^29."""
    n, bs, hkv = 2 ** 29 - 1, 19, 8
    v = torch.tensor([1, -1, 0, 1]).repeat(32)
    dtype = torch.bfloat16 if kv == "bf16" else torch.int8
    pools = dict(k_cache=torch.randint(-3, 4, (1, hkv, 128, 128)).to(dtype).cuda(),
                 v_cache=v.expand(1, hkv, 128, 128).contiguous().to(dtype).cuda())
    if kv == "int8":
        pools |= {x: torch.ones((1, hkv, 128), device="cuda") for x in ("k_scale", "v_scale")}
    out = torch.full((bs, hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((bs, hkv), 7.0, device="cuda")
    pages = 2 ** 22
    B.pa_tree_attention(q=torch.zeros((bs, hkv, 128), dtype=torch.bfloat16, device="cuda"),
                        page_table=torch.zeros((1, pages), dtype=torch.int32, device="cuda").repeat(bs, 1),
                        cache_seqlens=torch.full((bs,), n, dtype=torch.int32, device="cuda"),
                        cu_seqlens_q=torch.arange(bs + 1, dtype=torch.int32, device="cuda"),
                        tree_mask=torch.ones((bs, 1), dtype=torch.int64, device="cuda"), max_q_len=1,
                        max_seq_pages=pages, sm_scale=SCALE, out=out, lse=lse,
                        workspace=torch.empty(B.pa_tree_workspace_bytes(bs, bs, 1, hkv, hkv, 128, 128, pages),
                                              dtype=torch.uint8, device="cuda"), **pools)
    torch.cuda.synchronize()
    assert B.pa_read_error_flags(reset=True) == 0
    assert bool((out.cpu().double() == v).all())
    assert float((lse.cpu().double() - math.log(n)).abs().max()) <= 2.0 ** -20 * math.log(n)


# ---- lse ------------------------------------------------------------------------------------------


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("splits", [1, 3])
def test_tree_lse_is_good_to_fp32(kv, splits):
    """Small scores, so that little hides behind them.  A score: products of two bf16 (or a code) are
    exact, 128 truncating adds, the scales' and the softmax scale's rounding (132 * 2^-23 of
    sum |q k|).  A weight: the difference to the reference and 2^x, 2^-21.  l: n adds of positive
    terms, 2^-24 each at most.  ln l, m ln 2 and their sum: 2^-22 of |lse| + 1."""
    c = Cache([1500, 333, 129], 2, 64, kv, 35)
    t = Tree(c, [20, 5, 1], 8, 36)
    t.q *= 0.0625
    _, want, _ = R.tree_attention(t.q, c.k, c.v, c.ks, c.vs, c.table, c.n, t.q_lens, t.masks, SCALE)
    _, lse = t.run(splits)
    at = 0
    for b, (n, ql) in enumerate(zip(c.n, t.q_lens)):
        for h in range(8):
            k = R.pool_rows(c.k, c.ks, c.table[b], n, h // 4).abs()
            size = (t.q[at:at + ql, h].double().abs() @ k.T).amax(-1) * SCALE
            w = want[at:at + ql, h]
            bound = 132 * 2.0 ** -23 * size + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -22 * (w.abs() + 1)
            err = (lse[at:at + ql, h].cpu().double() - w).abs()
            assert bool((err <= bound).all()), (float(err.max()), float(bound.max()))
        at += ql


# ---- NaN scores --------------------------------------------------------------------------------


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("nodes", [6, 40])
def test_tree_nan_query_gives_nan(kv, splits, nodes):
    """A query with NaN gets NaN (out and lse), however its context is cut; one that sees nothing
    still gets 0 and -inf; the others keep their bits."""
    c = Cache([900, 20], 2, 64, kv, 31)
    masks = [m for p in ([-1] * nodes, [-1] * nodes) for m in R.ancestor_rows(p)]
    masks[nodes + 1] = 0
    t = Tree(c, [nodes, min(nodes, 20)], 16, 32, masks=masks[:nodes + min(nodes, 20)])
    clean = t.run(splits)
    t.q[2, 5, 7] = math.nan                              # one head of one query
    t.q[nodes + 3, 0, 0] = math.nan
    out, lse = t.run(splits)
    for row, head in ((2, 5), (nodes + 3, 0)):
        assert bool(torch.isnan(out[row, head]).all()) and bool(torch.isnan(lse[row, head]))
        out[row, head], lse[row, head] = clean[0][row, head], clean[1][row, head]
    assert same_bits(out, clean[0]) and same_bits(lse, clean[1])


@pytest.mark.parametrize("splits", [1, 6])
def test_tree_nan_key_of_a_committed_position_gives_nan(splits):
    """A NaN key far from the others' pieces reaches every query of its kv head and no other."""
    c = Cache([1500], 2, 64, "bf16", 33)
    t = Tree(c, [3], 4, 34)
    clean = t.run(splits)
    c.d_k[int(c.table[0, 0]), 1, 5] = math.nan
    out, lse = t.run(splits)
    assert bool(torch.isnan(out[:, 2:]).all()) and bool(torch.isnan(lse[:, 2:]).all())
    assert same_bits(out[:, :2], clean[0][:, :2]) and same_bits(lse[:, :2], clean[1][:, :2])


# ---- page tables wider than the lengths need ----------------------------------------------------


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("seqlens", [[900, 400, 77], [2000] * 5, [5000]])
def test_tree_cuts_do_not_depend_on_the_tables_width(kv, seqlens):
    """The same pieces (their sums in the workspace) and the same bits from a table of the
    longest request's width and from one sized for contexts 64 times as long."""
    c = Cache(seqlens, 4, 64, kv, 21)
    t = Tree(c, [5] * len(seqlens), 16, 22)
    wide = torch.full((len(seqlens), 64 * c.msp), -1, dtype=torch.int32)
    wide[:, :c.msp] = c.table
    splits, rows = 6, t.total * 16 * 6
    start = -(-rows * 4 // 256) * 256                    # m, then l, each on 256 bytes
    got = []
    for table, msp in ((c.d_table, c.msp), (wide.cuda(), 64 * c.msp)):
        ws = torch.full((B.pa_workspace_bytes(t.total, 16, 128, splits),), 255, dtype=torch.uint8, device="cuda")
        out, lse = t.run(splits, page_table=table, max_seq_pages=msp, workspace=ws)
        t.check(out, lse)
        got.append((out, lse, ws[start:start + rows * 4].view(torch.int32)))
    for a, b in zip(*got):
        assert same_bits(a, b)
    if len(seqlens) == 1:                                # (four units over the whole device: cut)
        assert bool((got[1][2].view(torch.float32).view(-1, splits)[:, 0] >= 0).all())


@pytest.mark.parametrize("kv,hq", [("bf16", 8), ("int8", 8), ("bf16", 32)])
def test_weights_do_not_depend_on_the_tables_width(kv, hq):
    """Blocks with one run of tokens and with several give the same bits: a row gets one sum."""
    seqlens = [3000, 1, 700, 2049]
    c = Cache(seqlens, 2, 64, kv, 23)
    q = torch.randn((4, hq, 128), generator=c.g).to(torch.bfloat16).cuda()
    lse = torch.full((4, hq), 6.0, device="cuda")
    got = []
    for width in (c.msp, 4096, 65536):
        table = torch.full((4, width), -1, dtype=torch.int32)
        table[:, :c.msp] = c.table
        w = c.d_w.clone()
        B.pa_accumulate_weights(q=q, lse=lse, k_cache=c.d_k, k_scale=c.d_ks, page_table=table.cuda(),
                                cache_seqlens=c.d_n, weights=w, max_seq_pages=width, sm_scale=SCALE)
        got.append(w)
    want, bound = R.accumulate(c.weights, q.cpu(), lse.cpu(), c.k, c.ks, c.table, seqlens, SCALE)
    assert bool(((got[0].cpu().double() - want).abs() <= bound).all())
    assert same_bits(got[0], got[1]) and same_bits(got[0], got[2])


def test_weights_of_long_contexts_in_several_runs():
    """Requests that reach past the first run of every block."""
    c = Cache([150001, 140000], 1, 128, "int8", 24)
    q = torch.randn((2, 4, 128), generator=c.g).to(torch.bfloat16)
    lse = torch.full((2, 4), 6.0)
    table = torch.full((2, 16 * c.msp), -1, dtype=torch.int32)
    table[:, :c.msp] = c.table
    B.pa_accumulate_weights(q=q.cuda(), lse=lse.cuda(), k_cache=c.d_k, k_scale=c.d_ks, page_table=table.cuda(),
                            cache_seqlens=c.d_n, weights=c.d_w, max_seq_pages=16 * c.msp, sm_scale=SCALE)
    want, bound = R.accumulate(c.weights, q, lse, c.k, c.ks, c.table, c.n, SCALE)
    assert bool(((c.d_w.cpu().double() - want).abs() <= bound).all())


def test_weights_time_does_not_follow_the_tables_width():
    """Short contexts under a table for a million tokens: no more than three times as long as under
    a table of their own (1.1 times; 9 with a block for each run of the table)."""
    bs, hkv, page, n = 32, 8, 64, 4096
    pool = torch.zeros((n // page * 2, hkv, page, 128), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(pool.shape[:3], device="cuda")
    q = torch.zeros((bs, 4 * hkv, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((bs, 4 * hkv), device="cuda")
    lens = torch.full((bs,), n, dtype=torch.int32, device="cuda")
    times = []
    for width in (n // page, (1 << 20) // page):
        table = torch.zeros((bs, width), dtype=torch.int32, device="cuda")
        table[:, :n // page] = torch.arange(n // page, device="cuda")
        call = B.prepare_accumulate_weights(q=q, lse=lse, k_cache=pool, page_table=table, cache_seqlens=lens,
                                            weights=w, max_seq_pages=width, sm_scale=SCALE)
        runs = []
        for _ in range(5):
            start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            for _ in range(20):
                call()
            stop.record()
            torch.cuda.synchronize()
            runs.append(start.elapsed_time(stop))
        times.append(sorted(runs)[2])
    assert times[1] < 3 * times[0], times


# ---- empty lists ---------------------------------------------------------------------------------


def test_compact_of_an_empty_list_only_writes_the_lengths():
    """Nothing accepted anywhere: a list of no columns (whose tensor has no memory)."""
    c = Cache([100, 30], 2, 64, "bf16", 41, poison=False)
    before = [dev.clone() for _, dev in c.pools()]
    new = torch.full((2,), 99, dtype=torch.int32, device="cuda")
    B.pa_compact_cache(page_table=c.d_table, cache_seqlens=c.d_n,
                       kept=torch.empty((2, 1, 0), dtype=torch.int32, device="cuda"),
                       counts=torch.zeros(2, dtype=torch.int32, device="cuda"),
                       begin=torch.tensor([95, 28], dtype=torch.int32).cuda(), k_cache=c.d_k, v_cache=c.d_v,
                       weights=c.d_w, max_seq_pages=c.msp, new_seqlens=new)
    assert new.tolist() == [95, 28]
    for a, (_, dev) in zip(before, c.pools()):
        assert same_bits(a, dev)
