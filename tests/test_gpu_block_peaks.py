"""Attention over a block-scaled cache where one token outweighs all others: what the small weights
add up to has to survive, against the float64 definition."""

import math

import pytest
import torch

import block_reference as R
from paged_kv_decode_metadata_gb300 import binding as B
from paged_kv_decode_metadata_gb300 import build
from test_gpu_block_cache import HALF_STEP, SCALE, BlockCache, attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    B.load()
    B.pa_read_error_flags(reset=True)
    yield
    assert B.pa_read_error_flags(reset=True) == 0


def peaked(n, hkv, group, new, page, block, gap, at, v_of_peak, seed, spread=0):
    """A request whose token `at` scores about `gap` above the others' mean for every query; its
    V row is 0 or like the others'.  The others' scores are normal, of standard deviation 1.
    ``spread``: V scales up to 2^spread apart."""
    c = BlockCache([n], hkv, page, block, seed)
    c.ks.fill_(0.01)
    base = torch.randn((hkv, 128), generator=c.g).clamp(-2.5, 2.5)
    q = (base[None, :, None] + 0.1 * torch.randn((new, hkv, group, 128), generator=c.g)).to(torch.bfloat16)
    # s ks c |base|^2 = gap
    codes = base * (gap / (SCALE * 0.01 * (base * base).sum(-1, keepdim=True)))
    p, r = int(c.table[0, at // page]), at % page
    c.k[p, :, r] = codes.clamp(-448, 448).to(torch.float8_e4m3fn)
    if v_of_peak == 0:
        c.v[p, :, r] = torch.zeros((hkv, 128)).to(torch.float8_e4m3fn)
    if spread:
        c.vs.mul_(torch.exp2(-torch.randint(0, spread + 1, c.vs.shape, generator=c.g).float()))
    c.to_device()
    return c, q.flatten(1, 2)


def check_peaked(c, q, out, lse):
    """Weights are rounded to fp16, 2^-11 sum p |v|, and what they are cut into ends 2^-36 below the
    chunk's largest V scale times the largest weight so far; scores and sums in 32 bits as in
    test_gpu_block_cache.check."""
    n, (new, hq) = c.n[0], q.shape[:2]
    group = hq // c.hkv
    o, ls, mass, size = R.attention(q, c.k, c.v, c.ks, c.vs, c.table, [n], [new], SCALE)
    chunk = torch.arange(n) // 128
    least = torch.zeros_like(o)
    for h in range(c.hkv):
        k, v = (R.rows(x, s, c.table[0], n, h) for x, s in ((c.k, c.ks), (c.v, c.vs)))
        scale = c.vs.double()[c.table[0].long()[torch.arange(n) // c.page], h, torch.arange(n) % c.page // c.block]
        tops = torch.zeros(int(chunk[-1]) + 1, dtype=torch.float64).scatter_reduce(0, chunk, scale, "amax")[chunk]
        codes = (tops / scale)[:, None] * v.abs()
        for i in range(new):
            seen = n - new + i + 1
            heads = slice(h * group, (h + 1) * group)
            x = q[i, heads].double() @ k[:seen].T * SCALE
            least[i, heads] = torch.exp(x.amax(-1) - ls[i, heads])[:, None] * codes[:seen].sum(0)
    bound = HALF_STEP * o.abs() + (2.0 ** -11 + 2.0 ** -18 + 2.0 ** -18 * size[..., None]) * mass + 2.0 ** -36 * least
    off = (out.double().cpu() - o).abs() / bound
    assert off.max() <= 1, f"out off by {off.max():.3g} of its bound"
    lim = 2.0 ** -19 * size + 2.0 ** -18 + 2.0 ** -22 * ls.abs()
    assert ((lse.double().cpu() - ls).abs() <= lim).all()
    return float((out.double().cpu() - o).abs().max() / o.abs().max())


@pytest.mark.parametrize("n,at", [(8192, 0), (8192, 5000), (8192, 8100), (131072, 0), (131072, 77777)])
@pytest.mark.parametrize("gap", [10, 14, 16, 18, 20])
@pytest.mark.parametrize("v_of_peak", [0, 1])
def test_one_token_outweighs_the_others(n, at, gap, v_of_peak):
    c, q = peaked(n, 1, 2, 1, 64, 64, gap, at, v_of_peak, seed=gap + at)
    out, lse = attend(c, q.cuda())
    rel = check_peaked(c, q, out, lse)
    # what is left is about the outputs' own rounding, not the weights': the bound above is met by
    # an output of zeros where sum p |v| is large beside it, this one is not
    assert rel <= 2.0 ** -7


@pytest.mark.parametrize("hkv,group,new,page,block", [(2, 1, 1, 16, 16), (1, 8, 1, 128, 32), (2, 4, 3, 32, 16),
                                                      (1, 16, 1, 64, 64), (2, 5, 5, 16, 16), (1, 32, 1, 128, 128),
                                                      (1, 8, 9, 64, 32)])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_every_tile_keeps_small_weights(hkv, group, new, page, block, splits):
    for gap, v_of_peak in ((19, 0), (15, 1)):
        c, q = peaked(3001, hkv, group, new, page, block, gap, 1234, v_of_peak, seed=page + group + gap)
        out, lse = attend(c, q.cuda(), [new], num_splits=splits)
        assert check_peaked(c, q, out, lse) <= 2.0 ** -7


@pytest.mark.parametrize("splits", [1, 4])
def test_small_weights_of_small_scales(splits):
    """V scales up to 2^12 apart within a chunk, beside a token that outweighs the rest."""
    c, q = peaked(2500, 2, 4, 2, 64, 16, 14, 700, 0, seed=5, spread=12)
    out, lse = attend(c, q.cuda(), [2], num_splits=splits)
    assert check_peaked(c, q, out, lse) <= 2.0 ** -7


@pytest.mark.parametrize("e", [-110, -60, 60, 110])
def test_v_scales_of_any_size(e):
    """Outputs scale with V: the same weights whatever the power of two."""
    c, q = peaked(700, 1, 8, 1, 64, 32, 12, 300, 1, seed=9)
    small, lse = attend(c, q.cuda(), num_splits=1)
    c.vs.mul_(2.0 ** e)
    c.to_device()
    out, again = attend(c, q.cuda(), num_splits=1)
    assert torch.equal(lse, again)
    assert torch.equal(out.double(), small.double() * 2.0 ** e)
    assert math.isfinite(float(out.float().abs().max()))


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("splits", [1, 2])
def test_scales_that_are_not_finite(bad, splits):
    """A K scale reaches the queries that see its block, a V scale no other request and no other head."""
    c = BlockCache([300, 300, 300], 2, 64, 16, 31)
    q = torch.randn((9, 8, 128), generator=c.g).to(torch.bfloat16)
    plain, _ = attend(c, q.cuda(), [3, 3, 3], num_splits=splits)
    page = int(c.table[0, 299 // 64])
    c.ks[page, 0, 299 % 64 // 16] = bad            # positions 288 .. 299: every query sees some
    c.vs[int(c.table[1, 1]), 1, 2] = bad
    c.to_device()
    out, lse = attend(c, q.cuda(), [3, 3, 3], num_splits=splits)
    gone = torch.zeros((9, 8), dtype=torch.bool)
    gone[:3, :4] = gone[3:6, 4:] = True
    assert torch.equal(~torch.isfinite(out.float()).all(-1).cpu(), gone)
    assert torch.equal(out.cpu()[~gone].view(torch.int16), plain.cpu()[~gone].view(torch.int16))
    # (V leaves the sums alone)
    assert bool(torch.isfinite(lse[3:]).all())
