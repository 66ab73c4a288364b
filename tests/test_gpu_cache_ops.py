"""GPU parity of the cache operators (rotary append, tree attention, accumulated weights,
compaction, eviction) against the float64 definitions in cache_reference.py."""

import math
import random

import pytest
import torch

import cache_reference as R
from paged_kv_decode_metadata_gb300 import binding as B
from paged_kv_decode_metadata_gb300 import build

pytestmark = pytest.mark.gpu

SCALE = float(torch.tensor(128 ** -0.5, dtype=torch.float32))
HALF_STEP = 2.0 ** -8      # bf16: a rounding is off by at most this, relative


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    B.load()
    B.pa_read_error_flags(reset=True)
    yield
    assert B.pa_read_error_flags(reset=True) == 0


class Cache:
    """Pools, page table and lengths of a batch, on the CPU and on the device.  Values past
    a request's length (and pages that no request owns) are NaN in bf16 pools."""

    def __init__(self, seqlens, hkv, page, kv, seed, extra_pages=3, poison=True):
        g = torch.Generator().manual_seed(seed)
        self.g, self.n, self.hkv, self.page, self.kv = g, list(seqlens), hkv, page, kv
        per = [-(-n // page) for n in seqlens]
        self.msp = max(max(per), 1)
        self.num_pages = sum(per) + extra_pages
        order = torch.randperm(self.num_pages, generator=g, dtype=torch.int32)
        self.table = torch.full((len(per), self.msp), 0, dtype=torch.int32)
        at = 0
        for b, c in enumerate(per):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.free = order[at:]
        shape = (self.num_pages, hkv, page, 128)
        if kv == "bf16":
            self.k, self.v = (torch.randn(shape, generator=g).to(torch.bfloat16) for _ in "kv")
            self.ks = self.vs = None
            if poison:
                owned = torch.zeros(shape[0], page, dtype=torch.bool)
                for b, n in enumerate(seqlens):
                    for j in range(n):
                        owned[self.table[b, j // page].item(), j % page] = True
                for x in (self.k, self.v):
                    x.masked_fill_(~owned[:, None, :, None], math.nan)
        else:
            self.k, self.v = (torch.randint(-127, 128, shape, generator=g, dtype=torch.int8) for _ in "kv")
            self.ks, self.vs = (torch.rand(shape[:3], generator=g) * 0.045 + 0.005 for _ in "kv")
        self.weights = torch.rand(shape[:3], generator=g)
        dev = lambda t: None if t is None else t.cuda()
        self.d_table, self.d_k, self.d_v, self.d_ks, self.d_vs, self.d_w = map(
            dev, (self.table, self.k, self.v, self.ks, self.vs, self.weights))
        self.d_n = torch.tensor(self.n, dtype=torch.int32).cuda()

    def pools(self):
        """(cpu, device) pairs of everything that travels with a row."""
        pairs = [(self.k, self.d_k), (self.v, self.d_v), (self.weights, self.d_w)]
        return pairs + ([(self.ks, self.d_ks), (self.vs, self.d_vs)] if self.kv == "int8" else [])


def same_bits(a, b):
    """Equal bit for bit (NaNs included)."""
    view = {2: torch.int16, 4: torch.int32, 1: torch.int8}[a.element_size()]
    return torch.equal(a.cpu().contiguous().view(view), b.cpu().contiguous().view(view))


# ---- rotary append --------------------------------------------------------------------------

ROPE_CASES = [  # tokens, hq, hkv, page, kv, rot, interleaved, amplitude, start, in_place, wide
    (1, 1, 1, 16, "bf16", 128, False, 1.0, 0, False, False),
    (1, 32, 8, 64, "int8", 128, False, 1.0, 131071, False, True),
    (7, 8, 2, 32, "bf16", 64, False, 1.25, 500, True, False),
    (33, 16, 16, 16, "int8", 32, True, 1.0, 7, False, True),
    (129, 12, 3, 128, "bf16", 16, True, 0.9, 10 ** 6, False, True),
    (65, 40, 8, 64, "bf16", 112, False, 1.0, 2 ** 31, True, False),
    (50, 64, 8, 64, "int8", 96, False, 1.3466, 999999, False, True),
    (1030, 4, 2, 64, "bf16", 128, True, 1.0, 3, False, True),
    (1500, 9, 1, 16, "int8", 128, False, 1.0, 60000, False, False),
]


@pytest.mark.parametrize("tokens,hq,hkv,page,kv,rot,inter,amp,start,in_place,wide", ROPE_CASES)
def test_rope_append(tokens, hq, hkv, page, kv, rot, inter, amp, start, in_place, wide):
    g = torch.Generator().manual_seed(tokens * 7 + rot)
    c = Cache([tokens], hkv, page, kv, tokens + rot, poison=False)
    qkv = torch.randn((tokens, hq + 2 * hkv, 128), generator=g).to(torch.bfloat16)
    pos = start + torch.randperm(tokens, generator=g)
    at = torch.randperm(tokens, generator=g)
    slots = c.table[0].long()[at // page] * page + at % page
    if tokens > 3:
        slots[2] = -1                                   # a padded token
        slots[tokens - 1] = -7
    freq = B.pa_rope_frequencies(rot, 10000.0, B.PA_ROPE_BY_PARTS, factor=8.0, original_length=2048,
                                 low=1.0, high=32.0)
    dev = qkv.cuda()
    parts = dev.split([hq, hkv, hkv], dim=1)
    q, k, v = parts if wide else (x.contiguous() for x in parts)
    out = q if in_place else torch.full((tokens, hq, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    B.pa_rope_append(q=q, k=k, v=v, positions=pos.cuda(), slots=slots.cuda(), inv_freq=freq.cuda(),
                     interleaved=inter, amplitude=amp, q_out=out, k_cache=c.d_k, v_cache=c.d_v,
                     k_scale=c.d_ks, v_scale=c.d_vs)
    torch.cuda.synchronize()
    cq, ck, cv = qkv.split([hq, hkv, hkv], dim=1)
    want_q, want_k = (R.rope(x, pos, freq, inter, amp) for x in (cq, ck))
    # fp32 rotation: sine and cosine to 2^-22 absolute, two products, one sum, the amplitude
    # (|a| + |b| <= twice the row's largest value), then one bf16 rounding
    big = lambda x: x.double().abs().amax(-1, keepdim=True)
    arith = lambda x: 2.0 ** -20 * max(amp, 1.0) * 2 * big(x)
    err = (out.cpu().double() - want_q).abs()
    assert bool((err <= HALF_STEP * (want_q.abs() + arith(cq)) + arith(cq)).all()), err.max()
    for cpu, devpool, scale, dscale, want, src in ((c.k, c.d_k, c.ks, c.d_ks, want_k, ck),
                                                   (c.v, c.d_v, c.vs, c.d_vs, cv.double(), cv)):
        got, touched = devpool.cpu(), torch.zeros(cpu.shape[0], page, dtype=torch.bool)
        tol = arith(src) if src is ck else 0.0 * big(src)
        for t in range(tokens):
            s = int(slots[t])
            if s < 0:
                continue
            touched[s // page, s % page] = True
            row = got[s // page, :, s % page].double()
            if kv == "bf16":
                bound = HALF_STEP * (want[t].abs() + tol[t]) + tol[t]
                assert bool(((row - want[t]).abs() <= bound).all())
            else:
                sc = dscale.cpu()[s // page, :, s % page].double()[:, None]
                top = want[t].abs().amax(-1, keepdim=True)
                # the largest magnitude / 127, one division
                assert bool(((sc - top / 127).abs() <= tol[t] / 127 + 2.0 ** -23 * top / 127).all())
                # half a step, the arithmetic, and x / scale rounded (127 * 2^-22 steps)
                assert bool(((row * sc - want[t]).abs() <= sc * (0.5 + 127 * 2.0 ** -22) + tol[t]).all())
                assert int(got[s // page, :, s % page].abs().max()) <= 127
        for h in range(hkv):                             # nothing else was written
            assert same_bits(got[:, h][~touched], cpu[:, h][~touched])
            if scale is not None:
                assert same_bits(dscale.cpu()[:, h][~touched], scale[:, h][~touched])
    if not in_place:
        assert same_bits(dev, qkv)                       # inputs are only read


@pytest.mark.parametrize("power", [-125, -110, -61, 100])
def test_rope_int8_codes_of_tiny_and_large_rows(power):
    """1 / scale of the smallest rows does not fit fp32."""
    c = Cache([3], 2, 16, "int8", 6)
    g = torch.Generator().manual_seed(9)
    x = (torch.randn((3, 2, 128), generator=g).double() * 2.0 ** power).to(torch.bfloat16)
    slots = int(c.table[0, 0]) * 16 + torch.arange(3)
    d = x.cuda()
    B.pa_rope_append(q=d, k=d, v=d, positions=torch.zeros(3, dtype=torch.int64).cuda(), slots=slots.cuda(),
                     inv_freq=B.pa_rope_frequencies(128).cuda(), q_out=torch.empty_like(d), k_cache=c.d_k,
                     v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs)
    page = int(c.table[0, 0])
    for pool, scales in ((c.d_k, c.d_ks), (c.d_v, c.d_vs)):   # (position 0 turns nothing)
        code = pool.cpu()[page, :, :3].double().transpose(0, 1)
        scale = scales.cpu()[page, :, :3].double().T[..., None]
        top = x.double().abs().amax(-1, keepdim=True)
        # one fp32 division, subnormal results within half of 2^-149
        assert bool(((scale - top / 127).abs() <= 2.0 ** -23 * top / 127 + 2.0 ** -150).all())
        # half a step, and 1 / scale and the product rounded (127 * 2^-22 steps)
        assert bool(((code * scale - x.double()).abs() <= scale * (0.5 + 127 * 2.0 ** -22)).all())


def test_rope_zero_row_and_slot_past_the_pool():
    c = Cache([20], 2, 16, "int8", 5)
    x = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([int(c.table[0, 0]) * 16 + 3, c.num_pages * 16]).cuda()
    before = c.d_k.clone()
    B.pa_rope_append(q=x, k=x, v=x, positions=torch.tensor([5, 6]).cuda(), slots=slots,
                     inv_freq=B.pa_rope_frequencies(128).cuda(), q_out=torch.empty_like(x), k_cache=c.d_k,
                     v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs)
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_SLOT_OUT_OF_RANGE
    page = int(c.table[0, 0])
    assert int(c.d_k[page, :, 3].abs().max()) == 0 and float(c.d_ks[page, :, 3].abs().max()) == 0
    before[page, :, 3] = 0
    assert torch.equal(c.d_k, before)


def test_append_before_a_step_with_pdl():
    """rotary append -> decode step, launched back to back with PDL, as a layer does: the
    step reads the rotated q before its own wait and the appended rows after it."""
    seq, hq, hkv, page = [700, 64, 1, 333], 8, 2, 64
    outs = []
    for pdl in (True, False):
        c = Cache(seq, hkv, page, "bf16", 11, poison=False)
        g = torch.Generator().manual_seed(12)
        x = torch.randn((4, hq + 2 * hkv, 128), generator=g).to(torch.bfloat16).cuda()
        q, k, v = x.split([hq, hkv, hkv], dim=1)
        last = torch.tensor(seq) - 1
        slots = (c.table.long()[torch.arange(4), last // page] * page + last % page).cuda()
        r2t = torch.zeros((4, c.msp * page), dtype=torch.int32)
        for b, n in enumerate(seq):
            j = torch.arange(n)
            r2t[b, :n] = c.table[b][j // page] * page + (j % page).int()
        q_out = torch.zeros((4, hq, 128), dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(q_out)
        lse = torch.zeros((4, hq), device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        ws = torch.empty(B.pa_workspace_bytes(4, hq, 128, 3), dtype=torch.uint8, device="cuda")
        step = dict(req_pool_indices=torch.arange(4).cuda(), seq_lens=torch.tensor(seq).cuda(),
                    req_to_token=r2t.cuda(), seqlen_offset=0, max_seq_pages=c.msp,
                    cache_seqlens=torch.empty(4, **i32), cu_seqlens_k=torch.empty(5, **i32),
                    page_table=torch.empty((4, c.msp), **i32), q=q_out, k_cache=c.d_k, v_cache=c.d_v,
                    num_splits=3, sm_scale=SCALE, workspace=ws, out=out, lse=lse, use_pdl=pdl)
        pos, freq = last.cuda(), B.pa_rope_frequencies(128).cuda()
        torch.cuda.synchronize()
        B.pa_rope_append(q=q, k=k, v=v, positions=pos, slots=slots, inv_freq=freq, q_out=q_out,
                         k_cache=c.d_k, v_cache=c.d_v, use_pdl=pdl)
        B.pa_decode_step(**step)
        torch.cuda.synchronize()
        c.k, c.v = c.d_k.cpu(), c.d_v.cpu()
        want, want_lse, mag = R.tree_attention(q_out.cpu(), c.k, c.v, None, None, c.table, seq, [1] * 4,
                                               [1] * 4, SCALE)
        assert bool(((out.cpu().double() - want).abs() <= 1e-2 + HALF_STEP * want.abs()).all())
        assert bool(((lse.cpu().double() - want_lse).abs() <= 1e-3).all())
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# ---- tree attention --------------------------------------------------------------------------


def random_parents(r, n):
    return [-1 if i == 0 or r.random() < 0.1 else r.randint(max(0, i - 9), i - 1) for i in range(n)]


class Tree:
    def __init__(self, cache, q_lens, hq, seed, masks=None):
        r = random.Random(seed)
        self.c, self.q_lens, self.hq = cache, list(q_lens), hq
        self.total = sum(q_lens)
        self.parents = [random_parents(r, n) for n in q_lens]
        self.masks = masks if masks is not None else [m for p in self.parents for m in R.ancestor_rows(p)]
        self.max_q = max(max(q_lens), 1)
        self.words = -(-self.max_q // 64)
        g = torch.Generator().manual_seed(seed)
        self.q = torch.randn((self.total, hq, 128), generator=g).to(torch.bfloat16)
        self.cu = torch.tensor([sum(q_lens[:i]) for i in range(len(q_lens) + 1)], dtype=torch.int32)

    def run(self, splits=0, pad=0, pdl=True, stream=None, **over):
        c = self.c
        rows = self.total + pad
        q = torch.zeros((rows, self.hq, 128), dtype=torch.bfloat16)
        q[:self.total] = self.q
        mask = torch.full((rows, self.words), -1, dtype=torch.int64)
        mask[:self.total] = R.mask_tensor(self.masks, self.words)
        out = torch.full((rows, self.hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((rows, self.hq), 7.0, device="cuda")
        s = splits or B.pa_choose_tree_splits(len(self.q_lens), self.max_q, self.hq, c.hkv, c.page, c.msp)
        ws = torch.full((max(B.pa_workspace_bytes(rows, self.hq, 128, s), 16),), 255, dtype=torch.uint8,
                        device="cuda")            # (NaN partials where nothing is written)
        kw = dict(q=q.cuda(), k_cache=c.d_k, v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs,
                  page_table=c.d_table, cache_seqlens=c.d_n, cu_seqlens_q=self.cu.cuda(),
                  tree_mask=mask.cuda(), max_q_len=self.max_q, max_seq_pages=c.msp, num_splits=splits,
                  sm_scale=SCALE, workspace=ws, out=out, lse=lse, use_pdl=pdl, stream=stream)
        kw.update(over)
        torch.cuda.synchronize()
        B.pa_tree_attention(**kw)
        torch.cuda.synchronize()
        return kw["out"], kw["lse"]

    def check(self, out, lse):
        c = self.c
        want, want_lse, mag = R.tree_attention(self.q, c.k, c.v, c.ks, c.vs, c.table, c.n, self.q_lens,
                                               self.masks, SCALE)
        out, lse = out[:self.total].cpu().double(), lse[:self.total].cpu().double()
        # each weight (int8: times its V scale) rounds to bf16 once, 2^-8 of its share of
        # sum p |V|; 2^-13 of it for the fp32 parts (scores, exponentials, sums); then the
        # output's own rounding
        e = (HALF_STEP + 2.0 ** -13) * mag
        err = (out - want).abs()
        assert bool((err <= HALF_STEP * (want.abs() + e) + e).all()), float((err - e).max())
        empty = torch.isinf(want_lse)
        assert torch.equal(torch.isneginf(lse), empty)
        assert bool((out[empty] == 0).all())
        assert bool(((lse - want_lse)[~empty].abs() <= 1e-3).all())


TREE_CASES = [  # seqlens, q_lens, hq, hkv, page, kv, splits
    ([1], [1], 1, 1, 16, "bf16", 0),
    ([5], [5], 4, 1, 64, "bf16", 1),
    ([64, 1, 130], [3, 1, 8], 8, 2, 64, "bf16", 1),
    ([300, 17, 64, 1000], [16, 0, 5, 33], 16, 4, 16, "bf16", 3),
    ([257, 128, 129], [32, 32, 32], 32, 8, 128, "bf16", 2),
    ([700, 300], [70, 129], 8, 1, 32, "bf16", 0),
    ([513, 640, 40], [64, 17, 40], 16, 2, 64, "bf16", 1),
    ([300], [256], 16, 1, 64, "bf16", 2),
    ([1000, 2000], [9, 4], 4, 4, 64, "bf16", 40),
    ([1], [1], 2, 1, 16, "int8", 1),
    ([300, 17, 64, 1000], [16, 0, 5, 33], 16, 4, 16, "int8", 3),
    ([513, 640, 40], [64, 17, 40], 16, 2, 64, "int8", 1),
    ([700, 129], [129, 100], 32, 2, 128, "int8", 0),
    ([260, 31], [13, 31], 3, 3, 32, "int8", 2),
]


@pytest.mark.parametrize("seqlens,q_lens,hq,hkv,page,kv,splits", TREE_CASES)
def test_tree_attention(seqlens, q_lens, hq, hkv, page, kv, splits):
    t = Tree(Cache(seqlens, hkv, page, kv, sum(seqlens)), q_lens, hq, sum(q_lens) + hq)
    t.check(*t.run(splits))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("splits", [1, 3])
def test_tree_empty_rows_padding_and_short_caches(kv, splits):
    """Rows whose mask leaves nothing; a request with more drafted than cached tokens; padded
    rows behind the batch, left as they were; a request with an empty cache."""
    c = Cache([4, 200, 0, 3], 2, 64, kv, 77)
    masks = [0, 1, 0, 0b1010] + [0] * 6 + [0] * 2 + [0b1000, 0b0011, 0b1111, 0b0100, 0]
    t = Tree(c, [4, 6, 2, 5], 4, 78, masks=masks)
    out, lse = t.run(splits, pad=9)
    t.check(out, lse)
    assert bool((out[t.total:] == 7.0).all()) and bool((lse[t.total:] == 7.0).all())


def test_tree_masked_keys_may_hold_anything():
    """NaN and infinities in the K rows of drafted positions that a query does not see."""
    c = Cache([150], 1, 64, "bf16", 5)
    page, row = int(c.table[0, 149 // 64]), 149 % 64
    masks = [1 << i for i in range(9)] + [1]            # the last position: seen by none
    for bad in (math.nan, math.inf, -math.inf):
        c.k[page, :, row] = bad
        c.d_k.copy_(c.k)
        t = Tree(c, [10], 8, 6, masks=masks)
        t.check(*t.run(1))


def test_tree_far_from_zero_scores():
    """Scores in the hundreds: the running maximum moves, nothing overflows."""
    c = Cache([600, 300], 2, 64, "bf16", 15)
    t = Tree(c, [20, 7], 8, 16)
    t.q *= 40
    want, want_lse, mag = R.tree_attention(t.q, c.k, c.v, None, None, c.table, c.n, t.q_lens, t.masks, SCALE)
    out, lse = t.run(2)
    # fp32 scores of magnitude up to S are off by 128 * 2^-24 * S, relative in the weights
    k_abs = torch.nan_to_num(c.k.double()).abs().amax()
    size = float(t.q.double().abs().sum(-1).max() * k_abs * SCALE)
    e = (HALF_STEP + 2 * 132 * 2.0 ** -24 * size) * mag
    assert bool(((out.cpu().double() - want).abs() <= HALF_STEP * (want.abs() + e) + e).all())
    assert bool(((lse.cpu().double() - want_lse).abs() <= 132 * 2.0 ** -24 * size + 1e-3).all())


def test_tree_pdl_streams_and_repeats_give_the_same_bits():
    c = Cache([900, 400, 77], 2, 64, "bf16", 21)
    t = Tree(c, [20, 40, 3], 16, 22)
    for splits in (1, 4):
        a = t.run(splits)
        for b in (t.run(splits), t.run(splits, pdl=False), t.run(splits, stream=torch.cuda.Stream())):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tree_page_out_of_range_sets_the_flag():
    c = Cache([300], 1, 64, "bf16", 31, poison=False)
    t = Tree(c, [4], 4, 32)
    for bad in (-1, c.num_pages, 2 ** 31 - 1):
        table = c.d_table.clone()
        table[0, 2] = bad
        t.run(1, page_table=table)
        assert B.pa_read_error_flags(reset=True) == B.DEVERR_PAGE_OUT_OF_RANGE
    t.run(1, cache_seqlens=torch.tensor([10 ** 6], dtype=torch.int32).cuda())
    assert B.pa_read_error_flags(reset=True) & B.DEVERR_SEQLEN_OUT_OF_RANGE
    for cu in ([0, 100], [-3, 1], [0, -1], [3, 9]):     # rows outside the batch: nothing is run
        out, _ = t.run(1, cu_seqlens_q=torch.tensor(cu, dtype=torch.int32).cuda())
        assert B.pa_read_error_flags(reset=True) == B.DEVERR_SEQLEN_OUT_OF_RANGE
        assert bool((out == 7.0).all())
    t.check(*t.run(1))


def test_tree_masks_from_parents():
    r = random.Random(3)
    q_lens = [1, 0, 64, 65, 256, 7]
    parents = [random_parents(r, n) for n in q_lens]
    want = R.mask_tensor([m for p in parents for m in R.ancestor_rows(p)], 5)
    cu = torch.tensor([sum(q_lens[:i]) for i in range(7)], dtype=torch.int32).cuda()
    flat = torch.tensor([x for p in parents for x in p] + [-1] * 4, dtype=torch.int32).cuda()
    got = torch.full((flat.numel(), 5), 99, dtype=torch.int64, device="cuda")
    B.pa_build_tree_mask(flat, cu, got, max_q_len=256)
    assert torch.equal(got[:-4].cpu(), want) and bool((got[-4:] == 99).all())
    flat[1 + 3] = 3                                       # a node that is its own parent
    B.pa_build_tree_mask(flat, cu, got, max_q_len=256)
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_TREE_PARENT
    assert got[1 + 3].tolist() == [8, 0, 0, 0, 0]


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_tree_step_and_chain_against_the_multi_query_step(kv):
    """pa_decode_step_tree: its metadata, and, for chains, pa_decode_step_multi's answer."""
    seq, hq, hkv, page = [300, 77, 64], 8, 2, 32
    c = Cache(seq, hkv, page, kv, 41)
    q_lens = [4, 2, 3]
    chain = [(1 << (i + 1)) - 1 for n in q_lens for i in range(n)]
    t = Tree(c, q_lens, hq, 42, masks=chain)
    r2t = torch.zeros((5, c.msp * page), dtype=torch.int32)
    rpi = torch.tensor([4, 0, 2])
    for b, n in enumerate(seq):
        j = torch.arange(n)
        r2t[rpi[b], :n] = c.table[b][j // page] * page + (j % page).int()
    i32 = dict(dtype=torch.int32, device="cuda")
    got = []
    for fn, extra in ((B.pa_decode_step_tree, dict(tree_mask=R.mask_tensor(chain, 1).cuda())),
                      (B.pa_decode_step_multi, {})):
        out = torch.zeros((9, hq, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((9, hq), device="cuda")
        meta = dict(cache_seqlens=torch.empty(3, **i32), cu_seqlens_k=torch.empty(4, **i32),
                    page_table=torch.empty((3, c.msp), **i32), cu_seqlens_q=torch.empty(4, **i32))
        fn(req_pool_indices=rpi.cuda(), seq_lens=torch.tensor(seq).cuda() - 1, req_to_token=r2t.cuda(),
           seqlen_offset=1, max_seq_pages=c.msp, q=t.q.cuda(), max_q_len=4, k_cache=c.d_k, v_cache=c.d_v,
           num_splits=3, sm_scale=SCALE, k_scale=c.d_ks, v_scale=c.d_vs, out=out, lse=lse,
           workspace=torch.empty(B.pa_workspace_bytes(9, hq, 128, 3), dtype=torch.uint8, device="cuda"),
           qlens=torch.tensor(q_lens).cuda(), q_mode=B.PA_Q_MODE_CUMSUM, **meta, **extra)
        torch.cuda.synchronize()
        t.check(out, lse)
        got.append({k: v.cpu() for k, v in meta.items()} | {"out": out, "lse": lse})
    for key in ("cache_seqlens", "cu_seqlens_k", "page_table", "cu_seqlens_q"):
        assert torch.equal(got[0][key], got[1][key])
    assert got[0]["cache_seqlens"].tolist() == seq
    assert bool(((got[0]["lse"] - got[1]["lse"]).abs() <= 2e-3).all())


def test_tree_captured_twice_and_replayed():
    """Two captured graphs, each with its own workspace, replayed on two streams at once,
    with new inputs in the same buffers."""
    c = Cache([800, 500], 2, 64, "bf16", 51)
    trees, graphs, bufs = [], [], []
    for k in range(2):
        t = Tree(c, [30, 12], 8, 52 + k)
        ws = torch.empty(B.pa_workspace_bytes(t.total, 8, 128, 4), dtype=torch.uint8, device="cuda")
        out = torch.zeros((t.total, 8, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((t.total, 8), device="cuda")
        q = torch.zeros_like(out)
        kw = dict(q=q, k_cache=c.d_k, v_cache=c.d_v, page_table=c.d_table, cache_seqlens=c.d_n,
                  cu_seqlens_q=t.cu.cuda(), tree_mask=R.mask_tensor(t.masks, 1).cuda(), max_q_len=30,
                  max_seq_pages=c.msp, num_splits=4, sm_scale=SCALE, workspace=ws, out=out, lse=lse)
        B.pa_tree_attention(**kw)                      # attributes set before the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.pa_tree_attention(**kw)
        trees.append(t)
        graphs.append(graph)
        bufs.append((q, out, lse, kw))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for t, (q, out, lse, _) in zip(trees, bufs):
        q.copy_(t.q)
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for t, (q, out, lse, _) in zip(trees, bufs):
        t.check(out, lse)


@pytest.mark.parametrize("seed", range(12))
def test_tree_random_shapes(seed):
    r = random.Random(seed)
    bs, hkv, group = r.randint(1, 4), r.choice([1, 2, 3]), r.choice([1, 2, 4, 8, 16])
    seqlens = [r.randint(1, 500) for _ in range(bs)]
    q_lens = [min(n, r.choice([0, 1, r.randint(1, 40), r.randint(1, 130)])) for n in seqlens]
    if sum(q_lens) == 0:
        q_lens[0] = 1
    c = Cache(seqlens, hkv, r.choice([16, 32, 64, 128]), r.choice(["bf16", "int8"]), seed)
    t = Tree(c, q_lens, hkv * group, seed + 100)
    t.check(*t.run(r.randint(0, 5)))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("splits", [0, 1, 2])
@pytest.mark.parametrize("equal", [False, True])
def test_tree_many_requests(kv, splits, equal):
    """More requests than a warp has lanes: ragged ones, some with nothing drafted or cached, and
    equal ones in as many units as the device has SMs, which stay whole."""
    r = random.Random(7)
    if equal:
        seqlens, q_lens, hkv, group = [300] * 38, [9] * 38, 4, 4
    else:
        seqlens = [r.choice([0, 1, 128, r.randint(1, 700)]) for _ in range(100)]
        q_lens = [min(n, r.choice([0, 1, 5, r.randint(1, 50)])) for n in seqlens]
        q_lens[31] = q_lens[32] = q_lens[99] = 2         # (of an empty cache, too)
        hkv, group = 2, 8
    t = Tree(Cache(seqlens, hkv, 32, kv, 3), q_lens, hkv * group, 4)
    t.check(*t.run(splits))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_tree_short_requests_while_memory_is_busy(kv):
    """Requests of a chunk or two, several to a block, so that the last V tiles of two of them are
    on their way at once; copies on another stream make that take longer.  Every call gives
    the first one's bits."""
    r = random.Random(11)
    seqlens = [r.randint(1, 171) for _ in range(30)]
    q_lens = [min(n, r.randint(1, 58)) for n in seqlens]
    t = Tree(Cache(seqlens, 16, 64, kv, 12), q_lens, 64, 13)
    out, lse = t.run(0)
    t.check(out, lse)
    c, rows = t.c, t.total
    size = B.pa_tree_workspace_bytes(30, rows, t.max_q, 64, 16, 128, 64, c.msp)
    again = torch.empty_like(out), torch.empty_like(lse)
    call = B.prepare_tree_attention(
        q=t.q.cuda(), k_cache=c.d_k, v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs, page_table=c.d_table,
        cache_seqlens=c.d_n, cu_seqlens_q=t.cu.cuda(), tree_mask=R.mask_tensor(t.masks, t.words).cuda(),
        max_q_len=t.max_q, max_seq_pages=c.msp, num_splits=0, sm_scale=SCALE,
        workspace=torch.empty(max(16, size), dtype=torch.uint8, device="cuda"), out=again[0], lse=again[1])
    side = torch.cuda.Stream()
    a, b = (torch.zeros(1 << 30, dtype=torch.uint8, device="cuda") for _ in "ab")
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(side):
            for _ in range(4):
                b.copy_(a)
        for _ in range(50):                              # (beside the copies)
            call()
        assert same_bits(out, again[0]) and same_bits(lse, again[1])


# ---- accumulated weights -----------------------------------------------------------------------

WEIGHT_CASES = [  # seqlens, hq, hkv, page, kv
    ([1], 1, 1, 16, "bf16"), ([300, 0, 17, 64], 8, 2, 64, "bf16"), ([1000, 255, 256, 257], 16, 1, 16, "bf16"),
    ([700], 4, 4, 128, "bf16"), ([1], 8, 1, 32, "int8"), ([300, 0, 17, 64], 8, 2, 64, "int8"),
    ([1000, 255], 32, 2, 16, "int8"), ([513, 700], 12, 3, 128, "int8"),
]


@pytest.mark.parametrize("seqlens,hq,hkv,page,kv", WEIGHT_CASES)
def test_accumulate_weights(seqlens, hq, hkv, page, kv):
    c = Cache(seqlens, hkv, page, kv, sum(seqlens) + hq)
    q = torch.randn((len(seqlens), hq, 128), generator=c.g).to(torch.bfloat16)
    _, lse, _ = R.tree_attention(q, c.k, c.v, c.ks, c.vs, c.table, seqlens, [1 if n else 0 for n in seqlens],
                                 [1] * len(seqlens), SCALE) if 0 not in seqlens else (None, None, None)
    if lse is None:                                     # (an empty request has no query row above)
        lse = torch.full((len(seqlens), hq), -math.inf, dtype=torch.float64)
        for b, n in enumerate(seqlens):
            for h in range(hq if n else 0):
                k = R.pool_rows(c.k, c.ks, c.table[b], n, h // (hq // hkv))
                lse[b, h] = torch.logsumexp(k @ q[b, h].double() * SCALE, -1)
    lse = lse.float()
    if hq > 1:
        lse[0, 1] = -math.inf                           # a head that attended to nothing
    want = c.weights
    bound = torch.zeros_like(want, dtype=torch.float64)
    total = want.double()
    for _ in range(2):                                  # twice: totals add up
        B.pa_accumulate_weights(q=q.cuda(), lse=lse.cuda(), k_cache=c.d_k, k_scale=c.d_ks,
                                page_table=c.d_table, cache_seqlens=c.d_n, weights=c.d_w,
                                max_seq_pages=c.msp, sm_scale=SCALE)
        total, more = R.accumulate(total, q, lse, c.k, c.ks, c.table, seqlens, SCALE)
        bound += more
    err = (c.d_w.cpu().double() - total).abs()
    assert bool((err <= bound).all()), float((err - bound).max())
    seen = torch.zeros((c.num_pages, page), dtype=torch.bool)
    for b, n in enumerate(seqlens):
        j = torch.arange(n)
        seen[c.table[b].long()[j // page], j % page] = True
    for h in range(hkv):                                # other rows are left as they were
        assert same_bits(c.d_w[:, h].cpu()[~seen], c.weights[:, h][~seen])


def test_accumulate_weights_of_a_shared_page():
    """Two requests that share their first pages: both add to the shared rows."""
    c = Cache([200, 200], 1, 64, "bf16", 9, poison=False)
    c.table[1, :2] = c.table[0, :2]
    q = torch.randn((2, 4, 128), generator=c.g).to(torch.bfloat16)
    lse = torch.full((2, 4), 5.0)
    B.pa_accumulate_weights(q=q.cuda(), lse=lse.cuda(), k_cache=c.d_k, page_table=c.table.cuda(),
                            cache_seqlens=c.d_n, weights=c.d_w, max_seq_pages=c.msp, sm_scale=SCALE)
    want, bound = R.accumulate(c.weights, q, lse, c.k, None, c.table, [200, 200], SCALE)
    assert bool(((c.d_w.cpu().double() - want).abs() <= 2 * bound).all())


def test_accumulate_weights_page_out_of_range():
    c = Cache([200], 1, 64, "bf16", 10, poison=False)
    table = c.d_table.clone()
    table[0, 1] = c.num_pages + 5
    B.pa_accumulate_weights(q=torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda"),
                            lse=torch.zeros((1, 2), device="cuda"), k_cache=c.d_k, page_table=table,
                            cache_seqlens=c.d_n, weights=c.d_w, max_seq_pages=c.msp, sm_scale=SCALE)
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_PAGE_OUT_OF_RANGE


# ---- eviction and compaction -----------------------------------------------------------------------


def evict(c, budget, first, recent, in_place, pdl=True):
    bs = len(c.n)
    kept = torch.full((bs, c.hkv, budget), 99, dtype=torch.int32, device="cuda")
    new = torch.full((bs,), 99, dtype=torch.int32, device="cuda")
    dst = None
    if not in_place:
        need = -(-min(budget, max(max(c.n), 1)) // c.page)
        dst = c.free[:bs * need].view(bs, need).contiguous().cuda()
        if need * c.page < min(budget, c.msp * c.page):   # columns for the longest possible request
            dst = torch.cat([dst, dst[:, -1:]], 1)
    B.pa_evict(page_table=c.d_table, cache_seqlens=c.d_n, weights=c.d_w, k_cache=c.d_k, v_cache=c.d_v,
               k_scale=c.d_ks, v_scale=c.d_vs, max_seq_pages=c.msp, budget=budget, num_first=first,
               num_recent=recent, dst_page_table=dst, kept=kept, new_seqlens=new, use_pdl=pdl)
    torch.cuda.synchronize()
    return kept.cpu(), new.cpu(), (c.table if in_place else dst.cpu())


def check_evict(c, budget, first, recent, in_place):
    want = []
    for b, n in enumerate(c.n):
        j = torch.arange(n)
        p = c.table[b].long()[j // c.page]
        want.append([R.kept_positions(c.weights[p, h, j % c.page].tolist(), n, budget, first, recent)
                     for h in range(c.hkv)])
    kept, new, dst = evict(c, budget, first, recent, in_place)
    assert new.tolist() == [min(n, budget) for n in c.n]
    for b in range(len(c.n)):
        for h in range(c.hkv):
            assert kept[b, h].tolist() == want[b][h] + [-1] * (budget - len(want[b][h]))
    moved = R.move([cpu for cpu, _ in c.pools()], c.table, dst, want, [0] * len(c.n))
    for w, (_, dev) in zip(moved, c.pools()):
        assert same_bits(dev, w)


EVICT_CASES = [  # seqlens, hkv, page, kv, budget, first, recent
    ([1], 1, 16, "bf16", 1, 0, 0), ([0, 5, 40], 2, 16, "bf16", 8, 2, 3),
    ([300, 64, 1000, 999], 3, 64, "bf16", 100, 4, 32), ([300, 64, 1000], 2, 32, "int8", 77, 0, 0),
    ([500], 1, 128, "int8", 200, 100, 100), ([2100, 33], 2, 16, "bf16", 1111, 1, 0),
    ([200, 100], 2, 64, "bf16", 150, 0, 150), ([4000], 4, 64, "int8", 3999, 4, 64),
]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("seqlens,hkv,page,kv,budget,first,recent", EVICT_CASES)
def test_evict(seqlens, hkv, page, kv, budget, first, recent, in_place):
    spare = sum(-(-budget // page) + 1 for _ in seqlens)
    c = Cache(seqlens, hkv, page, kv, budget + sum(seqlens), extra_pages=spare)
    check_evict(c, budget, first, recent, in_place)


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_ties_zeros_negatives_and_nan(in_place):
    c = Cache([700, 650], 2, 64, "bf16", 61, extra_pages=20)
    pick = torch.tensor([0.0, -0.0, 1.0, 1.0, -2.5, math.nan, math.inf, -math.inf, 1e-42, 3.0])
    c.weights = pick[torch.randint(0, 10, c.weights.shape, generator=c.g)]
    c.d_w.copy_(c.weights)
    check_evict(c, 333, 3, 20, in_place)


def test_evict_equal_weights_keeps_the_lowest_positions():
    c = Cache([5000], 1, 64, "bf16", 62, extra_pages=4)
    c.weights.zero_()
    c.d_w.zero_()
    kept, new, _ = evict(c, 100, 0, 10, True)
    assert kept[0, 0].tolist() == list(range(90)) + list(range(4990, 5000)) and new.tolist() == [100]


def test_evict_row_longer_than_shared_memory_holds():
    n = 60001
    c = Cache([n], 1, 128, "int8", 63, extra_pages=40)
    check_evict(c, 4321, 4, 100, False)


def test_evict_in_place_on_captured_graph_matches_eager():
    runs = []
    for capture in (False, True):
        c = Cache([900, 333], 2, 64, "bf16", 64)
        kept = torch.zeros((2, 2, 128), dtype=torch.int32, device="cuda")
        new = torch.zeros(2, dtype=torch.int32, device="cuda")
        call = B.prepare_evict(page_table=c.d_table, cache_seqlens=c.d_n, weights=c.d_w, k_cache=c.d_k,
                               v_cache=c.d_v, max_seq_pages=c.msp, budget=128, num_recent=16, kept=kept,
                               new_seqlens=new, stream=None if not capture else None)
        if capture:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                B.pa_evict(page_table=c.d_table, cache_seqlens=c.d_n, weights=c.d_w, k_cache=c.d_k,
                           v_cache=c.d_v, max_seq_pages=c.msp, budget=128, num_recent=16, kept=kept,
                           new_seqlens=new)
            graph.replay()
        else:
            call()
        torch.cuda.synchronize()
        runs.append([x.cpu() for x in (kept, new, c.d_k, c.d_v, c.d_w)])
    for a, b in zip(*runs):
        assert same_bits(a, b)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_compact_keeps_an_accepted_path_in_place(kv):
    """The accepted nodes of each request's tree move up behind the committed positions; one
    list serves every head, and other rows stay as they were."""
    seq, q_len = [300, 64, 131, 90], [9, 9, 9, 1]
    paths = [[0, 2, 5, 8], [], [1, 2, 3], [0]]
    c = Cache(seq, 3, 32, kv, 71)
    begin = [n - q for n, q in zip(seq, q_len)]
    kept = torch.full((4, 1, 5), -1, dtype=torch.int32)
    for b, path in enumerate(paths):
        kept[b, 0, :len(path)] = torch.tensor([begin[b] + t for t in path], dtype=torch.int32)
    counts = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    new = torch.zeros(4, dtype=torch.int32, device="cuda")
    lists = [[[begin[b] + t for t in path]] * 3 for b, path in enumerate(paths)]
    want = R.move([cpu for cpu, _ in c.pools()], c.table, c.table, lists, begin)
    B.pa_compact_cache(page_table=c.d_table, cache_seqlens=c.d_n, kept=kept.cuda(), counts=counts.cuda(),
                       begin=torch.tensor(begin, dtype=torch.int32).cuda(), k_cache=c.d_k, v_cache=c.d_v,
                       k_scale=c.d_ks, v_scale=c.d_vs, weights=c.d_w, max_seq_pages=c.msp, new_seqlens=new)
    torch.cuda.synchronize()
    assert new.tolist() == [b + len(p) for b, p in zip(begin, paths)]
    for w, (_, dev) in zip(want, c.pools()):
        assert same_bits(dev, w)


def test_compact_refuses_positions_out_of_range():
    c = Cache([100], 1, 64, "bf16", 72, poison=False)
    before = [dev.clone() for _, dev in c.pools()]
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    for pos, at in ((100, 0), (-1, 0), (2 ** 31 - 1, 0), (4, 5), (4, -1), (4, 2 ** 31 - 1)):
        B.pa_compact_cache(page_table=c.d_table, cache_seqlens=c.d_n,
                           kept=torch.tensor([[[pos]]], dtype=torch.int32).cuda(), counts=one, begin=one * at,
                           k_cache=c.d_k, v_cache=c.d_v, max_seq_pages=c.msp)
        assert B.pa_read_error_flags(reset=True) == B.DEVERR_KEPT_OUT_OF_RANGE
    for a, (_, dev) in zip(before, c.pools()):
        assert same_bits(a, dev)


# ---- together ----------------------------------------------------------------------------------------


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_speculative_loop(kv):
    """Two rounds as a server runs them: the drafted tokens are rotated and appended, the
    trees verified, the accepted paths kept, then a decode token appended and attended to,
    its weights accumulated, and the caches shrunk in place.  Every stage's result is
    checked against the definitions on the pools as they stand."""
    hq, hkv, page, msp = 8, 2, 16, 24
    n = [200, 37]
    g = torch.Generator().manual_seed(81)
    r = random.Random(82)
    c = Cache([msp * page] * 2, hkv, page, kv, 83, poison=False)   # pages for growth
    c.d_w.zero_()
    freq = B.pa_rope_frequencies(64, 10000.0, B.PA_ROPE_LINEAR, factor=2.0)
    position = list(n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()

    def append(count):
        """Rotated and appended tokens; returns q rows.  n grows."""
        t = sum(count)
        x = torch.randn((t, hq + 2 * hkv, 128), generator=g).to(torch.bfloat16).cuda()
        q, k, v = x.split([hq, hkv, hkv], dim=1)
        where = [(b, n[b] + i) for b in range(2) for i in range(count[b])]
        slots = torch.tensor([int(c.table[b, j // page]) * page + j % page for b, j in where]).cuda()
        pos = torch.tensor([position[b] + j - n[b] for b, j in where]).cuda()
        q_out = torch.empty((t, hq, 128), dtype=torch.bfloat16, device="cuda")
        B.pa_rope_append(q=q, k=k, v=v, positions=pos, slots=slots, inv_freq=freq.cuda(), q_out=q_out,
                         k_cache=c.d_k, v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs)
        want = R.rope(q.cpu(), pos.cpu(), freq, False, 1.0)
        big = q.cpu().double().abs().amax(-1, keepdim=True) * 2.0 ** -19
        assert bool(((q_out.cpu().double() - want).abs() <= HALF_STEP * (want.abs() + big) + big).all())
        for b in range(2):
            n[b] += count[b]
        return q_out

    def attend(q, count, masks):
        t = Tree(c, count, hq, 0, masks=masks)
        t.q = q.cpu()
        c.n, c.d_n = list(n), i32(n)
        c.k, c.v = c.d_k.cpu(), c.d_v.cpu()
        c.ks, c.vs = (c.d_ks.cpu(), c.d_vs.cpu()) if kv == "int8" else (None, None)
        out, lse = t.run(0)
        t.check(out, lse)
        return lse

    for _ in range(2):
        count = [7, 5]
        parents = [random_parents(r, k) for k in count]
        q = append(count)
        attend(q, count, [m for p in parents for m in R.ancestor_rows(p)])
        path = []
        for p in parents:                                 # a root-to-node path
            node, nodes = len(p) - 1, []
            while node >= 0:
                nodes.append(node)
                node = p[node]
            path.append(nodes[::-1])
        begin = [a - b for a, b in zip(n, count)]
        kept = torch.full((2, 1, 7), -1, dtype=torch.int32)
        for b in range(2):
            kept[b, 0, :len(path[b])] = torch.tensor([begin[b] + t for t in path[b]])
        new = torch.empty(2, dtype=torch.int32, device="cuda")
        B.pa_compact_cache(page_table=c.d_table, cache_seqlens=i32(n), kept=kept.cuda(),
                           counts=i32([len(p) for p in path]), begin=i32(begin), k_cache=c.d_k,
                           v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs, weights=c.d_w,
                           max_seq_pages=msp, new_seqlens=new)
        n = new.tolist()
        assert n == [a + len(p) for a, p in zip(begin, path)]
        position = [p + len(x) for p, x in zip(position, path)]
        q = append([1, 1])
        lse = attend(q, [1, 1], [1, 1])
        c.weights = c.d_w.cpu()
        B.pa_accumulate_weights(q=q, lse=lse, k_cache=c.d_k, k_scale=c.d_ks, page_table=c.d_table,
                                cache_seqlens=c.d_n, weights=c.d_w, max_seq_pages=msp, sm_scale=SCALE)
        want, bound = R.accumulate(c.weights, q.cpu(), lse.cpu(), c.k, c.ks, c.table, n, SCALE)
        assert bool(((c.d_w.cpu().double() - want).abs() <= bound).all())
        c.weights = c.d_w.cpu()
        position = [p + 1 for p in position]
        check_evict(c, 60, 2, 20, True)
        n = [min(x, 60) for x in n]


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_pages_past_four_gigabytes_give_the_same_bits(kv):
    """Append, tree, weights and both moves on pages whose byte offsets pass 32 bits, against the
    same pages at the start of a small pool."""
    hq, hkv, page, m = 16, 8, 64, 12
    g = torch.Generator().manual_seed(91)
    size = 2 if kv == "bf16" else 1
    far = 2 ** 32 // (hkv * page * 128 * size) + 1
    dtype = torch.bfloat16 if kv == "bf16" else torch.int8
    shape = (m, hkv, page, 128)
    first = [torch.randn(shape, generator=g).to(dtype) if kv == "bf16" else
             torch.randint(-127, 128, shape, generator=g, dtype=dtype) for _ in "kv"]
    first += [torch.rand(shape[:3], generator=g) * 0.045 + 0.005 for _ in range(3)]  # scales, weights
    x = torch.randn((20, hq + 2 * hkv, 128), generator=g).to(torch.bfloat16).cuda()
    q, k, v = x.split([hq, hkv, hkv], dim=1)
    masks = R.mask_tensor([m for p in ([-1, 0, 0, 1, 2, -1, 5, 6, 7, 8], [-1] * 10) for m in R.ancestor_rows(p)], 1)
    cu = torch.tensor([0, 10, 20], dtype=torch.int32).cuda()
    n = torch.tensor([370, 129], dtype=torch.int32).cuda()
    freq = B.pa_rope_frequencies(128).cuda()
    results = []
    for off in (0, far):
        pools = [torch.empty((off + m, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in first]
        for big, small in zip(pools, first):
            big[off:] = small.cuda()
        pk, pv, ks, vs, w = pools
        ks, vs = (ks, vs) if kv == "int8" else (None, None)
        table = torch.tensor([[3, 7, 1, 0, 9, 11], [2, 10, 4, 5, 6, 8]], dtype=torch.int32) + off
        at = [(0, 360 + i) for i in range(10)] + [(1, 119 + i) for i in range(10)]
        slots = torch.tensor([int(table[b, j // page]) * page + j % page for b, j in at]).cuda()
        table = table.cuda()
        rows = dict(page_table=table, max_seq_pages=6)
        cache = dict(k_cache=pk, v_cache=pv, k_scale=ks, v_scale=vs)
        q_out = torch.empty((20, hq, 128), dtype=torch.bfloat16, device="cuda")
        B.pa_rope_append(q=q, k=k, v=v, positions=torch.arange(20).cuda(), slots=slots, inv_freq=freq,
                         q_out=q_out, **cache)
        out, lse = torch.empty_like(q_out), torch.empty((20, hq), device="cuda")
        ws = torch.empty(max(16, B.pa_tree_workspace_bytes(2, 20, 10, hq, hkv, 128, page, 6)),
                         dtype=torch.uint8, device="cuda")
        B.pa_tree_attention(q=q_out, cache_seqlens=n, cu_seqlens_q=cu, tree_mask=masks.cuda(), max_q_len=10,
                            num_splits=0, sm_scale=SCALE, workspace=ws, out=out, lse=lse, **rows, **cache)
        B.pa_accumulate_weights(q=q_out[9::10].contiguous(), lse=lse[9::10].contiguous(), k_cache=pk,
                                k_scale=ks, cache_seqlens=n, weights=w, sm_scale=SCALE, **rows)
        kept = torch.empty((2, hkv, 100), dtype=torch.int32, device="cuda")
        new = torch.empty(2, dtype=torch.int32, device="cuda")
        evict = dict(weights=w, budget=100, num_first=3, num_recent=20, kept=kept, new_seqlens=new, **rows, **cache)
        # the first request to the second's last pages, then both in place
        B.pa_evict(cache_seqlens=torch.tensor([370, 0], dtype=torch.int32).cuda(),
                   dst_page_table=(torch.tensor([[6, 8], [6, 8]], dtype=torch.int32) + off).cuda(), **evict)
        B.pa_evict(cache_seqlens=n, dst_page_table=table, **evict)
        torch.cuda.synchronize()
        results.append([t.cpu() for t in (q_out, out, lse, kept, new)] +
                       [t[off:].cpu() for t in (pk, pv, w) + ((ks, vs) if kv == "int8" else ())])
        del pools, pk, pv, ks, vs, w, cache, evict
    for near, there in zip(*results):
        assert same_bits(near, there)
