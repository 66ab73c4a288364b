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
    """Weights carry 12 bits (2^-12 sum p |v|).  Scores: the pieces' products are added in the
    tensor cores' 32 bits, 4 sums of 32, truncated: 2^-20 sum |q k| covers them, the pieces'
    2^-21 and the fp32 factors; a weight is off by twice that (numerator and sum).  Then the
    output's rounding."""
    o, ls, mass, size = ref
    got = out.double().cpu()
    bound = HALF_STEP * o.abs() + (2.0 ** -12 + 2.0 ** -18 + 2.0 ** -18 * size[..., None]) * mass + 1e-30
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
