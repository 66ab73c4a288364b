"""GPU parity of the block-scaled cache (append, attention, decode step) against the float64
definitions in block_reference.py."""

import math

import pytest
import torch

import block_reference as R
from paged_kv_decode_metadata_gb300 import binding as B
from paged_kv_decode_metadata_gb300 import build

pytestmark = pytest.mark.gpu

SCALE = float(torch.tensor(128 ** -0.5, dtype=torch.float32))
HALF_STEP = 2.0 ** -8      # bf16: a rounding is off by at most this, relative
NAN_CODE = 0x7f


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    B.load()
    B.pa_read_error_flags(reset=True)
    yield
    assert B.pa_read_error_flags(reset=True) == 0


class BlockCache:
    """Pools, page table and lengths of a batch, on the CPU and on the device.  Codes past a
    request's length, and the scales of blocks that no request reaches, are NaN."""

    def __init__(self, seqlens, hkv, page, block, seed, extra_pages=3):
        g = torch.Generator().manual_seed(seed)
        self.g, self.n, self.hkv, self.page, self.block = g, list(seqlens), hkv, page, block
        per = [-(-n // page) for n in seqlens]
        self.msp = max(max(per), 1)
        self.num_pages = sum(per) + extra_pages
        order = torch.randperm(self.num_pages, generator=g, dtype=torch.int32)
        self.table = torch.full((len(per), self.msp), 0, dtype=torch.int32)
        at = 0
        for b, c in enumerate(per):
            self.table[b, :c] = order[at:at + c]
            at += c
        shape = (self.num_pages, hkv, page, 128)
        owned = torch.zeros(self.num_pages, page, dtype=torch.bool)
        for b, n in enumerate(seqlens):
            for j in range(0, n, page):
                owned[self.table[b, j // page].item(), :min(page, n - j)] = True
        touched = owned.view(self.num_pages, page // block, block).any(-1)
        pools = []
        for _ in "kv":
            x = (torch.randn(shape, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
            x.view(torch.uint8)[~owned[:, None, :].expand(-1, hkv, -1)] = NAN_CODE
            s = torch.rand((self.num_pages, hkv, page // block), generator=g) * 0.015 + 0.005
            s[~touched[:, None].expand(-1, hkv, -1)] = math.nan
            pools += [x, s]
        self.k, self.ks, self.v, self.vs = pools
        self.to_device()
        self.d_table = self.table.cuda()
        self.d_n = torch.tensor(self.n, dtype=torch.int32).cuda()

    def to_device(self):
        self.d_k, self.d_ks, self.d_v, self.d_vs = (x.cuda() for x in (self.k, self.ks, self.v, self.vs))


def rows_of(q_lens):
    cu = torch.zeros(len(q_lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(q_lens), 0)
    return cu


def attend(c, q, q_lens=None, **kw):
    """pa_block_attention over the cache; out and lse are prefilled to see what is written."""
    total, hq, _ = q.shape
    mql = kw.pop("max_q_len", max(q_lens) if q_lens else 1)
    out = torch.full((total, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total, hq), 7.0, device="cuda")
    splits = kw.get("num_splits", 0) or B.pa_choose_block_splits(len(c.n), mql, hq, c.hkv, c.page, c.msp)
    ws = torch.full((B.pa_workspace_bytes(total, hq, 128, splits),), 0xff, dtype=torch.uint8, device="cuda")
    B.pa_block_attention(q=q, k_cache=c.d_k, v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs,
                         page_table=c.d_table, cache_seqlens=c.d_n,
                         cu_seqlens_q=rows_of(q_lens).cuda() if q_lens else None, max_q_len=mql,
                         max_seq_pages=c.msp, sm_scale=kw.pop("sm_scale", SCALE), out=out, lse=lse,
                         workspace=ws, **kw)
    torch.cuda.synchronize()
    return out, lse


def check(out, lse, ref, sm_scale=SCALE):
    """Weights are rounded to fp16 (2^-11 sum p |v|).  Scores: the pieces' products are added in the
    tensor cores' 32 bits, 4 sums of 32, truncated: 2^-20 sum |q k| covers them, the pieces'
    2^-21 and the fp32 factors; a weight is off by twice that (numerator and sum).  Then the
    output's rounding."""
    o, ls, mass, size = ref
    got = out.double().cpu()
    bound = HALF_STEP * o.abs() + (2.0 ** -11 + 2.0 ** -18 + 2.0 ** -18 * size[..., None]) * mass + 1e-30
    bad = (got - o).abs() > bound
    assert not bad.any(), f"out off by {((got - o).abs() / bound).max():.3g} of its bound"
    dead = ls == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, dead)
    off = (lse.double().cpu() - ls)[~dead].abs()
    lim = (2.0 ** -19 * size + 2.0 ** -18 + 2.0 ** -22 * ls.abs())[~dead]
    assert (off <= lim).all(), f"lse off by {(off / lim).max():.3g} of its bound"


CASES = [  # seqlens, q_lens (None: one query per request), hq, hkv, page, block, splits
    ([1], None, 1, 1, 16, 16, 0),
    ([1024], None, 32, 8, 64, 64, 0),
    ([127, 128, 129], None, 8, 8, 128, 128, 1),
    ([300, 1, 0, 513], None, 8, 1, 64, 32, 3),
    ([5, 70, 260], [5, 3, 1], 12, 4, 16, 16, 2),
    ([4, 0, 33], [4, 2, 7], 7, 1, 32, 16, 0),
    ([640, 1500], [9, 2], 10, 2, 32, 32, 0),
    ([2000], [16], 32, 2, 64, 16, 5),
    ([777, 31], [1, 1], 32, 1, 16, 16, 4),
    ([129, 400], [40, 3], 5, 5, 128, 64, 1),
    ([3, 260], [6, 5], 16, 1, 64, 64, 2),
    ([900], [1], 31, 1, 128, 32, 0),
]


@pytest.mark.parametrize("seqlens,q_lens,hq,hkv,page,block,splits", CASES)
def test_attention(seqlens, q_lens, hq, hkv, page, block, splits):
    c = BlockCache(seqlens, hkv, page, block, seed=hq + page + len(seqlens))
    lens = q_lens or [1] * len(seqlens)
    q = torch.randn((sum(lens), hq, 128), generator=c.g).to(torch.bfloat16)
    out, lse = attend(c, q.cuda(), q_lens, num_splits=splits)
    check(out, lse, R.attention(q, c.k, c.v, c.ks, c.vs, c.table, seqlens, lens, SCALE))


# ---- append -----------------------------------------------------------------------------------

APPEND_CASES = [  # seqlens, q_lens, hq, hkv, page, block, rot, interleaved, amplitude
    ([1], [1], 4, 1, 16, 16, 128, False, 1.0),
    ([200, 64, 65, 1], [1, 1, 1, 1], 32, 8, 64, 64, 128, False, 1.0),
    ([300, 129], [300, 70], 8, 2, 64, 32, 64, True, 1.25),
    ([90, 17, 40], [33, 17, 0], 6, 3, 16, 16, 16, False, 0.9),
    ([260, 500], [131, 129], 5, 5, 128, 128, 96, True, 1.0),
    ([1000], [999], 16, 2, 128, 16, 128, False, 1.0),
    ([50, 70], [20, 9], 0, 4, 32, 32, 0, False, 1.0),
    # few rows a request on average, up to 1, 4 and 8, some requests with more
    ([30, 100, 64, 17, 128, 5, 61, 33], [1, 0, 0, 3, 0, 0, 2, 1], 8, 4, 32, 32, 128, False, 1.0),
    ([70, 9, 300, 65, 2, 128], [5, 3, 4, 1, 2, 6], 40, 8, 64, 64, 64, True, 1.0),
    ([70, 9, 300, 65, 8, 128], [8, 8, 7, 6, 8, 11], 6, 2, 128, 16, 96, False, 1.1),
    ([500] * 3, [1, 1, 1], 5, 5, 128, 128, 128, True, 1.0),
]


def append_inputs(c, q_lens, hq, rot, seed):
    """New rows of every request; some requests' are large, some zero, some small."""
    g = torch.Generator().manual_seed(seed)
    rows = sum(q_lens)
    wide = torch.randn((rows, hq + 2 * c.hkv + 1, 128), generator=g)
    size = torch.tensor([1.0, 30.0, 2.0 ** -30, 0.0])[torch.arange(rows) // 7 % 4]
    wide = (wide * torch.where(size > 0, size, 0.0)[:, None, None]).to(torch.bfloat16)
    positions = torch.cat([torch.arange(n - d, n) for n, d in zip(c.n, q_lens)]) * 37 + seed
    inv = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))
    return wide, positions, inv


def run_append(c, q_lens, wide, positions, inv, hq, interleaved, amplitude, **kw):
    d_wide = wide.cuda()
    q, k, v, _ = d_wide.split([hq, c.hkv, c.hkv, 1], dim=1)
    q_out = torch.full((wide.shape[0], hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    rot = dict(positions=positions.cuda(), inv_freq=inv.cuda()) if inv.numel() else {}
    B.pa_rope_append_blocks(q=q if hq else None, q_out=q_out if hq else None, k=k, v=v,
                            k_cache=c.d_k, v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs,
                            cu_seqlens_q=kw.pop("cu", rows_of(q_lens)).cuda(),
                            cache_seqlens=c.d_n, page_table=c.d_table, max_seq_pages=c.msp,
                            interleaved=interleaved, amplitude=amplitude, **rot, **kw)
    torch.cuda.synchronize()
    return q_out


def near_codes(got, want, exact_x, scale):
    """Codes equal but where the value lies within 2^-18 of a border between two codes (the
    fp32 rotation: sines to 2 ulp, two products and a sum: below 6 * 2^-23 of the largest term)."""
    off = got != want
    if not off.any():
        return
    gap = (got - want).abs()[off]
    assert (gap <= torch.maximum(want.abs()[off], got.abs()[off]) * 2.0 ** -3 + 2.0 ** -9).all()
    middle = (got + want)[off] / 2
    x = (exact_x / scale)[off]
    assert ((x - middle).abs() <= 2.0 ** -18 * 448).all()
    assert off.double().mean() < 1e-3


@pytest.mark.parametrize("seqlens,q_lens,hq,hkv,page,block,rot,interleaved,amplitude", APPEND_CASES)
def test_append(seqlens, q_lens, hq, hkv, page, block, rot, interleaved, amplitude):
    c = BlockCache(seqlens, hkv, page, block, seed=rot + page)
    for s in (c.ks, c.vs):  # as earlier appends leave them: powers of two, some too small
        s.copy_(torch.exp2(-torch.randint(3, 12, s.shape, generator=c.g).float()))
    c.to_device()
    wide, positions, inv = append_inputs(c, q_lens, hq, rot, seed=page)
    q_out = run_append(c, q_lens, wide, positions, inv, hq, interleaved, amplitude)
    q, k, v, _ = wide.split([hq, hkv, hkv, 1], dim=1)
    turn = (lambda x: R.rope(x, positions, inv, interleaved, amplitude)) if rot else (lambda x: x.double())
    if hq:
        want = turn(q)
        pair = want.abs().amax(-1, keepdim=True)
        assert ((q_out.double().cpu() - want).abs() <= HALF_STEP * want.abs() + 2.0 ** -20 * pair).all()
    for x, codes, scale, d_codes, d_scale in ((turn(k), c.k, c.ks, c.d_k, c.d_ks),
                                              (v.double(), c.v, c.vs, c.d_v, c.d_vs)):
        want, ws = R.code_values(codes), scale.double()
        before = want.clone()
        at = 0
        values = before.clone() * ws.repeat_interleave(block, -1)[..., None]
        for b, (n, d) in enumerate(zip(seqlens, q_lens)):
            if d:
                R.append(x[at:at + d], want, ws, c.table[b], n)
                for i in range(d):
                    j = n - d + i
                    values[int(c.table[b, j // page]), :, j % page] = x[at + i]
            at += d
        assert torch.equal(d_scale.cpu().double(), ws)
        got = R.code_values(d_codes.cpu())
        # (rows that nothing wrote hold what they held, NaN codes among them)
        same = torch.isnan(want)
        assert torch.equal(torch.isnan(got), same)
        full = torch.where(ws > 0, ws, 1.0).repeat_interleave(block, -1)[..., None].expand_as(want)
        zero = torch.zeros(())
        near_codes(torch.where(same, zero, got), torch.where(same, zero, want),
                   torch.where(same, zero, values), full)
        again = d_codes.clone()
    # the same append once more leaves the same bits
    run_append(c, q_lens, wide, positions, inv, hq, interleaved, amplitude)
    assert torch.equal(c.d_v.view(torch.uint8), again.view(torch.uint8))


# ---- the contract around the numbers --------------------------------------------------------------


def raw_call(c, q, out, lse, cu, mql, **kw):
    splits = kw.pop("num_splits", 0)
    ws = torch.full((B.pa_workspace_bytes(q.shape[0], q.shape[1], 128, max(splits, 70)),), 0xff, dtype=torch.uint8,
                    device="cuda")
    return B.prepare_block_attention(
        q=q, k_cache=c.d_k, v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs, page_table=kw.pop("table", c.d_table),
        cache_seqlens=kw.pop("n", c.d_n), cu_seqlens_q=cu, max_q_len=mql, max_seq_pages=kw.pop("msp", c.msp),
        sm_scale=SCALE, out=out, lse=lse, workspace=ws, num_splits=splits, **kw)


def blank(rows, hq):
    return (torch.full((rows, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((rows, hq), 7.0, device="cuda"))


def same(a, b):
    return torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32),
                       b.view(torch.int16 if b.element_size() == 2 else torch.int32))


@pytest.mark.parametrize("hq,hkv,splits", [(8, 2, 1), (8, 2, 3), (32, 2, 0), (32, 1, 2)])
def test_rows_that_no_request_covers_stay(hq, hkv, splits):
    """Padding rows, rows before the first request and those of refused requests."""
    c = BlockCache([300, 40, 20, 700], hkv, 64, 32, 71)
    q = torch.randn((14, hq, 128), generator=c.g).to(torch.bfloat16)
    out, lse = blank(14, hq)
    cu = torch.tensor([2, 4, 9, 9, 11], dtype=torch.int32).cuda()    # the second has 5 > max_q_len
    raw_call(c, q.cuda(), out, lse, cu, 4, num_splits=splits)()
    torch.cuda.synchronize()
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_SEQLEN_OUT_OF_RANGE
    ref = R.attention(torch.cat((q[2:4], q[9:11])), c.k, c.v, c.ks, c.vs, c.table[[0, 3]], [300, 700], [2, 2], SCALE)
    pick = [2, 3, 9, 10]
    check(out[pick], lse[pick], ref)
    rest = [i for i in range(14) if i not in pick]
    assert bool((out[rest] == 7.0).all()) and bool((lse[rest] == 7.0).all())


@pytest.mark.parametrize("splits", [1, 3])
def test_a_query_that_sees_nothing(splits):
    """Queries before the context's start, and an empty context."""
    c = BlockCache([3, 0, 200], 2, 16, 16, 72)
    q = torch.randn((7 + 2 + 5, 6, 128), generator=c.g).to(torch.bfloat16)
    out, lse = attend(c, q.cuda(), [7, 2, 5], num_splits=splits)
    check(out, lse, R.attention(q, c.k, c.v, c.ks, c.vs, c.table, c.n, [7, 2, 5], SCALE))
    assert not out[:4].any() and bool((lse[:4] == -math.inf).all())
    assert not out[7:9].any() and bool((lse[7:9] == -math.inf).all())


def test_non_finite_values_stay_where_they_are_seen():
    c = BlockCache([150, 150], 2, 64, 64, 73)
    q = torch.randn((6, 8, 128), generator=c.g).to(torch.bfloat16)
    q[4, 3, 77] = math.nan
    q[5, 6, 0] = math.inf
    page, row = int(c.table[0, 149 // 64]), 149 % 64     # the first request's newest token
    c.k.view(torch.uint8)[page, 1, row, 5] = NAN_CODE     # seen by its last query alone, heads 4 .. 7
    c.to_device()
    out, lse = attend(c, q.cuda(), [3, 3], num_splits=2)
    bad = torch.isnan(out.float()).all(-1).cpu()
    want = torch.zeros(6, 8, dtype=torch.bool)
    want[2, 4:] = want[4, 3] = want[5, 6] = True
    assert torch.equal(bad, want) and torch.equal(torch.isnan(lse).cpu(), want)
    assert torch.equal(torch.isnan(out.float()).any(-1).cpu(), want)


def test_blocks_of_zeros_and_of_very_different_scales():
    """Zero scales (rows of zeros as the append leaves them); scales 2^12 apart in one chunk."""
    c = BlockCache([256, 130], 1, 64, 16, 74)
    for s in (c.ks, c.vs):
        s.copy_(torch.exp2(torch.randint(-12, 1, s.shape, generator=c.g).float()))
    for b, n in enumerate(c.n):
        for j in range(16 * b, n, 48):
            p, i = int(c.table[b, j // 64]), j % 64 // 16
            c.ks[p, 0, i] = c.vs[p, 0, i] = 0.0
    c.to_device()
    q = (torch.randn((2, 4, 128), generator=c.g) * 0.02).to(torch.bfloat16)
    out, lse = attend(c, q.cuda(), num_splits=1)
    check(out, lse, R.attention(q, c.k, c.v, c.ks, c.vs, c.table, c.n, [1, 1], SCALE))
    c.vs.zero_()
    c.to_device()
    out, again = attend(c, q.cuda(), num_splits=3)
    assert not out.any() and torch.allclose(lse, again, rtol=0, atol=1e-4)


@pytest.mark.parametrize("factor", [1e30, 1e-30, 65536.0])
def test_queries_of_any_size(factor):
    c = BlockCache([200], 2, 64, 64, 75)
    q = (torch.randn((1, 8, 128), generator=c.g) * factor).to(torch.bfloat16)
    scale = SCALE / factor
    out, lse = attend(c, q.cuda(), num_splits=1, sm_scale=scale)
    check(out, lse, R.attention(q, c.k, c.v, c.ks, c.vs, c.table, c.n, [1], scale), scale)


def test_what_the_device_alone_sees_is_reported():
    c = BlockCache([100, 90], 2, 16, 16, 76)
    q = torch.randn((2, 4, 128), generator=c.g).to(torch.bfloat16).cuda()
    out, lse = blank(2, 4)
    table = c.d_table.clone()
    table[0, 2] = c.num_pages
    table[1, 1] = -3
    raw_call(c, q, out, lse, None, 1, table=table)()
    torch.cuda.synchronize()
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_PAGE_OUT_OF_RANGE
    n = torch.tensor([c.msp * 16 + 1, -5], dtype=torch.int32).cuda()
    raw_call(c, q, out, lse, None, 1, n=n)()
    torch.cuda.synchronize()
    assert B.pa_read_error_flags(reset=True) & B.DEVERR_SEQLEN_OUT_OF_RANGE
    assert not out[1].any() and bool((lse[1] == -math.inf).all())


def test_equal_inputs_give_equal_bits_whatever_the_pages_and_the_launch():
    c = BlockCache([1000, 13, 400], 4, 32, 16, 77)
    q = torch.randn((9, 16, 128), generator=c.g).to(torch.bfloat16).cuda()
    first = attend(c, q, [4, 3, 2])
    for pdl in (True, False):
        again = attend(c, q, [4, 3, 2], use_pdl=pdl)
        assert same(first[0], again[0]) and same(first[1], again[1])
    # a wider table, pages in another order
    perm = torch.randperm(c.num_pages, generator=c.g)
    for x, d in ((c.k, "d_k"), (c.v, "d_v"), (c.ks, "d_ks"), (c.vs, "d_vs")):
        moved = torch.empty_like(x)
        moved.view(torch.uint8)[perm] = x.view(torch.uint8)
        setattr(c, d, moved.cuda())
    c.d_table = perm.to(torch.int32)[c.table.long()].cuda()
    again = attend(c, q, [4, 3, 2])
    assert same(first[0], again[0]) and same(first[1], again[1])


def test_two_captured_graphs_with_their_own_workspaces():
    """Captured on a side stream, replayed in turn with other queries and lengths."""
    c = BlockCache([500, 900], 2, 64, 64, 78)
    side = torch.cuda.Stream()
    cases = []
    for k in range(2):
        q = torch.randn((2, 8, 128), generator=c.g).to(torch.bfloat16).cuda()
        out, lse = blank(2, 8)
        n = c.d_n.clone()
        with torch.cuda.stream(side):
            call = raw_call(c, q, out, lse, None, 1, num_splits=4 + k, n=n)
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                raw = raw_call(c, q, out, lse, None, 1, num_splits=4 + k, n=n)
                raw()
        cases.append((graph, q, out, lse, n, call, raw))
    for step in range(3):
        for k, (graph, q, out, lse, n, *_) in enumerate(cases):
            q.copy_(torch.randn((2, 8, 128), generator=c.g).to(torch.bfloat16))
            n.copy_(torch.tensor([500 - 130 * step, 900 - 77 * k - 1 * step], dtype=torch.int32))
        torch.cuda.synchronize()
        for graph, *_ in cases:
            graph.replay()
        torch.cuda.synchronize()
        for graph, q, out, lse, n, *_ in cases:
            lens = n.tolist()
            check(out, lse, R.attention(q.cpu(), c.k, c.v, c.ks, c.vs, c.table, lens, [1, 1], SCALE))


def test_pages_past_four_gigabytes():
    """Page and scale offsets past 2^32 bytes, in attention and append."""
    page, hkv = 128, 8
    pages = (5 << 30) // (hkv * page * 128) + 3
    pool = torch.empty((2, pages, hkv, page, 128), dtype=torch.uint8, device="cuda")
    c = BlockCache([300], hkv, page, 128, 79)
    c.table[0, :3] = torch.tensor([pages - 1, 5, pages - 2])
    big = []
    for i, (x, s) in enumerate(((c.k, c.ks), (c.v, c.vs))):
        used = (torch.randn((3, hkv, page, 128), generator=c.g) * 90).clamp(-448, 448).to(torch.float8_e4m3fn)
        scale = torch.full((pages, hkv, 1), math.nan)
        for j in range(3):
            pool[i, c.table[0, j].item()] = used[j].view(torch.uint8).cuda()
            scale[c.table[0, j].item()] = torch.rand((hkv, 1), generator=c.g) * 0.01 + 0.01
        big.append((used, scale))
    c.d_k, c.d_v = (pool[i].view(torch.float8_e4m3fn) for i in range(2))
    c.d_ks, c.d_vs = (s.cuda() for _, s in big)
    c.d_table, c.num_pages, c.msp = c.table.cuda(), pages, 3
    q = torch.randn((1, 32, 128), generator=c.g).to(torch.bfloat16)
    out, lse = attend(c, q.cuda())
    small = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    order = c.table[0].long()
    check(out, lse, R.attention(q, big[0][0], big[1][0], big[0][1][order], big[1][1][order], small, [300], [1], SCALE))
    new = torch.ones((1, hkv, 128), dtype=torch.bfloat16, device="cuda")
    n = torch.tensor([301], dtype=torch.int32).cuda()
    B.pa_rope_append_blocks(k=new, v=new * 2, k_cache=c.d_k, v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs,
                            cu_seqlens_q=torch.tensor([0, 1], dtype=torch.int32).cuda(), cache_seqlens=n,
                            page_table=c.d_table, max_seq_pages=3)
    torch.cuda.synchronize()
    got = pool[1, pages - 2, :, 300 - 256].view(torch.float8_e4m3fn).float() * c.d_vs[pages - 2]
    assert bool(((got - 2.0).abs() <= 2.0 * 2.0 ** -4).all())


def test_append_leaves_rows_of_refused_requests():
    c = BlockCache([100, 60, 30], 2, 16, 16, 80)
    wide, positions, inv = append_inputs(c, [4, 3, 2], 4, 128, 80)
    before = [x.clone() for x in (c.d_k, c.d_v, c.d_ks, c.d_vs)]
    table = c.d_table.clone()
    c.d_table[0, 6] = c.num_pages + 9                       # the page of positions 96 ..
    c.d_n = torch.tensor([100, 2, 30], dtype=torch.int32).cuda()   # fewer than its three new rows
    q_out = run_append(c, [4, 3, 2], wide, positions, inv, 4, False, 1.0)
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_PAGE_OUT_OF_RANGE | B.DEVERR_SEQLEN_OUT_OF_RANGE
    assert bool((q_out[4:7] == 7.0).all()) and not bool((q_out[7:] == 7.0).any())
    pages = [int(table[2, 28 // 16])]
    for x, y in zip(before, (c.d_k, c.d_v, c.d_ks, c.d_vs)):
        x, y = (z.view(torch.uint8) if z.element_size() == 1 else z.view(torch.int32) for z in (x, y))
        changed = (x != y).flatten(1).any(1).nonzero().flatten().tolist()
        assert set(changed) <= set(pages)


def test_append_in_place_on_a_projection_and_grown_scales():
    """q turned in place in the projection it lies in; a block filled token by token, larger and
    larger, holds what one append of all tokens would, to the halvings' rounding."""
    hkv, n = 2, 16
    c = BlockCache([n], hkv, 16, 16, 81)
    d = BlockCache([n], hkv, 16, 16, 81)
    wide = torch.randn((n, 4 + 2 * hkv, 128), generator=c.g)
    wide = (wide * torch.exp2(torch.arange(n).float() / 2)[:, None, None]).to(torch.bfloat16)
    inv = 10000.0 ** (-2.0 * torch.arange(64, dtype=torch.float64) / 128)
    whole, by_one = wide.cuda(), wide.cuda()
    def append(c, rows, lo, hi):
        q, k, v = rows[lo:hi].split([4, hkv, hkv], dim=1)
        B.pa_rope_append_blocks(q=q, q_out=q, k=k, v=v, positions=torch.arange(lo, hi).cuda(), inv_freq=inv.cuda(),
                                k_cache=c.d_k, v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs,
                                cu_seqlens_q=torch.tensor([0, hi - lo], dtype=torch.int32).cuda(),
                                cache_seqlens=torch.tensor([hi], dtype=torch.int32).cuda(), page_table=c.d_table,
                                max_seq_pages=c.msp)
    append(c, whole, 0, n)
    for i in range(n):
        append(d, by_one, i, i + 1)
    torch.cuda.synchronize()
    assert torch.equal(whole[:, :4].view(torch.int16), by_one[:, :4].view(torch.int16))
    want = R.rope(wide[:, :4], torch.arange(n), inv, False, 1.0)
    big = want.abs().amax(-1, keepdim=True)
    assert ((whole[:, :4].double().cpu() - want).abs() <= HALF_STEP * want.abs() + 2.0 ** -20 * big).all()
    p = int(c.table[0, 0])
    assert torch.equal(c.d_ks[p], d.d_ks[p]) and torch.equal(c.d_vs[p], d.d_vs[p])
    for x, y, s in ((c.d_k, d.d_k, c.d_ks), (c.d_v, d.d_v, c.d_vs)):
        a, b = x[p].float(), y[p].float()
        # a code is exact through a halving until it leaves the normal range: then each of up to 9
        # halvings rounds to the smallest step, 2^-9, by half of it at most, halved by the later ones
        assert bool(((a - b).abs() <= torch.where(a.abs() < 2.0 ** -6, 2.0 ** -9, 0.0)).all())


@pytest.mark.parametrize("q_lens,mql", [([1, 1, 1], 1), ([4, 1, 3], 4), ([1, 8, 5], 8), ([2, 7, 8], 8)])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 32), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_by_warps_and_by_thread_blocks_writes_the_same_bits(q_lens, mql, page, block, interleaved):
    """max_q_len picks the kernel: with the drafts' own length warps have the blocks, with a
    larger one thread blocks do."""
    seqlens = [page + 5, 2 * page + 3, max(page // 2, 8)]
    results = []
    for most in (mql, 60):
        c = BlockCache(seqlens, 2, page, block, 82)
        for s in (c.ks, c.vs):
            s.copy_(torch.exp2(-torch.randint(3, 12, s.shape, generator=c.g).float()))
        c.to_device()
        wide, positions, inv = append_inputs(c, q_lens, 6, 96, 82)
        wide, positions = (torch.cat([x, x.new_zeros((60 - len(x),) + x.shape[1:])]) for x in (wide, positions))
        q_out = run_append(c, q_lens, wide, positions, inv, 6, interleaved, 1.0, max_q_len=most)
        results.append([x.view(torch.uint8).clone() for x in (q_out, c.d_k, c.d_v, c.d_ks, c.d_vs)])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_append_of_a_prompt_among_decoding_requests():
    """Twenty requests with a row each and one with 130: every request's rows as by a call of its own."""
    seqlens, q_lens = [40 + i for i in range(20)] + [150], [1] * 20 + [130]
    c, d = (BlockCache(seqlens, 2, 64, 64, 83) for _ in range(2))
    wide, positions, inv = append_inputs(c, q_lens, 4, 128, 83)
    q_out = run_append(c, q_lens, wide, positions, inv, 4, False, 1.0)
    at, table, n = 0, d.d_table, d.d_n
    for b, rows in enumerate(q_lens):
        d.d_table, d.d_n = table[b:b + 1], n[b:b + 1]
        alone = run_append(d, [rows], wide[at:at + rows], positions[at:at + rows], inv, 4, False, 1.0)
        assert torch.equal(q_out[at:at + rows].view(torch.int16), alone.view(torch.int16))
        at += rows
    for a, b in zip((c.d_k, c.d_v, c.d_ks, c.d_vs), (d.d_k, d.d_v, d.d_ks, d.d_vs)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("q_lens,hq,hkv", [([5, 1, 1, 2, 4, 5], 10, 2), ([1, 8, 2, 10, 7, 1], 5, 1),
                                           ([2, 1, 0, 1, 2, 1], 16, 1), ([3, 1, 2, 1, 1, 3], 20, 2)])
def test_tiles_with_empty_columns_between_full_ones(q_lens, hq, hkv, splits):
    """Short drafts among longer ones and tiles of a remainder: columns 8, 16 or 24 to 31 of a
    tile are empty for some pieces of a block's share and not for the next."""
    seqlens = [300, 900, 2, 700, 129, 2000]
    c = BlockCache(seqlens, hkv, 64, 32, 84)
    q = torch.randn((sum(q_lens), hq, 128), generator=c.g).to(torch.bfloat16)
    out, lse = attend(c, q.cuda(), q_lens, num_splits=splits)
    check(out, lse, R.attention(q, c.k, c.v, c.ks, c.vs, c.table, seqlens, q_lens, SCALE))


def append_time(c, q_lens, max_q_len):
    """Microseconds of an append (32 / 8 heads), best of five replays of a graph of ten."""
    rows = sum(q_lens)
    wide, positions, inv = append_inputs(c, q_lens, 32, 128, 1)
    q, k, v, _ = wide.cuda().split([32, c.hkv, c.hkv, 1], dim=1)
    kw = dict(q=q, q_out=torch.empty((rows, 32, 128), dtype=torch.bfloat16, device="cuda"), k=k, v=v, k_cache=c.d_k,
              v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs, cu_seqlens_q=rows_of(q_lens).cuda(),
              cache_seqlens=c.d_n, page_table=c.d_table, max_seq_pages=c.msp, positions=positions.cuda(),
              inv_freq=inv.cuda(), max_q_len=max_q_len)
    side = torch.cuda.Stream()
    best = math.inf
    with torch.cuda.stream(side):
        B.pa_rope_append_blocks(**kw)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call = B.prepare_rope_append_blocks(**kw)
            for _ in range(10):
                call()
        graph.replay()
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
            a.record()
            graph.replay()
            b.record()
            side.synchronize()
            best = min(best, a.elapsed_time(b) * 100)
    return best


def test_a_prompt_in_a_padded_batch_is_not_appended_row_by_row():
    """200 rows of one request in a batch of 256 where all but two others have none, and max_q_len
    says so: within four times what the three take by themselves (a row at a time by single warps
    it is ten times)."""
    alone = append_time(BlockCache([300, 40, 41], 8, 64, 64, 85), [200, 1, 1], 200)
    padded = append_time(BlockCache([300, 40, 41] + [10] * 253, 8, 64, 64, 85), [200, 1, 1] + [0] * 253, 200)
    assert padded <= 4 * alone, (padded, alone)


@pytest.mark.parametrize("q_lens,mql", [([1] * 20, 4), ([1] * 20, 8), ([1] * 20, 15), ([13, 1] + [0] * 14 + [2], 13),
                                        ([18, 0, 1] + [0] * 22, 18), ([0, 30] + [1] * 6 + [0] * 30, 30)])
@pytest.mark.parametrize("page,block", [(16, 16), (128, 64)])
def test_append_of_sparse_batches_writes_the_same_bits(q_lens, mql, page, block):
    """Fewer rows than requests: whatever max_q_len makes of it, equal bits."""
    seqlens = [n + 3 * i for i, n in enumerate(q_lens)]
    results = []
    for most in (mql, 200):                                  # (200: the host knows nothing)
        c = BlockCache(seqlens, 2, page, block, 86)
        for s in (c.ks, c.vs):
            s.copy_(torch.exp2(-torch.randint(3, 12, s.shape, generator=c.g).float()))
        c.to_device()
        wide, positions, inv = append_inputs(c, q_lens, 6, 96, 86)
        q_out = run_append(c, q_lens, wide, positions, inv, 6, False, 1.0, max_q_len=most)
        results.append([x.view(torch.uint8).clone() for x in (q_out, c.d_k, c.d_v, c.d_ks, c.d_vs)])
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cu", [[0, 3, 100000, 100002], [0, 3, -900, -898], [500, 501, 502, 503], [0, 3, 3, 2000000000]])
@pytest.mark.parametrize("mql", [2, 3, 2000000000])
def test_append_reports_rows_far_outside(cu, mql):
    """Requests whose rows lie beyond every slot of the launch are refused and reported, too."""
    c = BlockCache([40, 41, 42], 2, 16, 16, 87)
    before = [x.clone() for x in (c.d_k, c.d_v, c.d_ks, c.d_vs)]
    wide, positions, inv = append_inputs(c, [3, 2, 2], 4, 128, 87)
    q_out = run_append(c, [3, 2, 2], wide, positions, inv, 4, False, 1.0, cu=torch.tensor(cu, dtype=torch.int32),
                       max_q_len=mql)
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_SEQLEN_OUT_OF_RANGE
    covered = 3 if cu[0] == 0 and mql >= 3 else 0
    assert bool((q_out[covered:] == 7.0).all())
    if not covered:
        for x, y in zip(before, (c.d_k, c.d_v, c.d_ks, c.d_vs)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_an_empty_request_with_more_than_32_gigabytes_of_rows():
    """Nothing cached and 65535 x 2080 rows of 256 bytes (q is not read, so out stands in for it)."""
    c = BlockCache([0], 65, 16, 16, 88)
    out = torch.full((65535, 65 * 32, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((65535, 65 * 32), 7.0, device="cuda")
    B.pa_block_attention(q=out, k_cache=c.d_k, v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs, page_table=c.d_table,
                         cache_seqlens=c.d_n, cu_seqlens_q=rows_of([65535]).cuda(), max_q_len=65535,
                         max_seq_pages=c.msp, sm_scale=SCALE, out=out, lse=lse, num_splits=1)
    torch.cuda.synchronize()
    assert bool((lse == -math.inf).all())
    for part in out.split(4096):
        assert not bool(part.view(torch.int16).any())


@pytest.mark.parametrize("seqlens,q_lens,hq,hkv,page,block,rot,interleaved,amplitude", APPEND_CASES)
def test_an_append_repeated_leaves_the_same_bits(seqlens, q_lens, hq, hkv, page, block, rot, interleaved, amplitude):
    """Keys, values, both scales and the turned queries, blocks with rows before the new ones among them."""
    c = BlockCache(seqlens, hkv, page, block, seed=rot + page)
    for s in (c.ks, c.vs):
        s.copy_(torch.exp2(-torch.randint(3, 12, s.shape, generator=c.g).float()))
    c.to_device()
    wide, positions, inv = append_inputs(c, q_lens, hq, rot, seed=page)
    first = run_append(c, q_lens, wide, positions, inv, hq, interleaved, amplitude)
    once = [x.clone() for x in (first, c.d_k, c.d_v, c.d_ks, c.d_vs)]
    again = run_append(c, q_lens, wide, positions, inv, hq, interleaved, amplitude)
    for a, b in zip(once, (again, c.d_k, c.d_v, c.d_ks, c.d_vs)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
