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
