"""The cache operators' host side: refusals of the C entry points and of the binding, the
rotary frequency tables, split counts (none of these calls reaches a GPU)."""

import math

import pytest
import torch

from paged_kv_decode_metadata_gb300 import binding as B
from paged_kv_decode_metadata_gb300 import build

FAKE = 1 << 20   # an aligned, never-dereferenced device address


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return B.load()


def _caller(fn, defaults):
    def call(**over):
        assert set(over) <= set(defaults), over
        return fn(*{**defaults, **over}.values())
    return call


ROPE = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, pos=FAKE, slots=FAKE, freq=FAKE, rot=128,
            inter=0, amp=1.0, tokens=3, hq=8, hkv=2, d=128, qo=FAKE + 4096, qos=1024, kc=FAKE, vc=FAKE,
            ksc=None, vsc=None, kv=0, P=64, pages=10, stream=None, pdl=1)


@pytest.mark.parametrize("over,status", [
    (dict(tokens=0), B.PA_OK),
    (dict(tokens=-1), B.PA_ERR_INVALID),
    (dict(q=None), B.PA_ERR_INVALID),
    (dict(slots=None), B.PA_ERR_INVALID),
    (dict(freq=None), B.PA_ERR_INVALID),
    (dict(q=FAKE + 8), B.PA_ERR_INVALID),          # misaligned rows
    (dict(ks=255), B.PA_ERR_INVALID),              # stride narrower than the heads
    (dict(qs=1028), B.PA_ERR_INVALID),             # rows off 16-byte boundaries
    (dict(qo=FAKE, qos=2048), B.PA_ERR_INVALID),   # in place with another stride
    (dict(amp=math.inf), B.PA_ERR_INVALID),
    (dict(kv=1), B.PA_ERR_INVALID),                # int8 without scales
    (dict(kv=2), B.PA_ERR_INVALID),
    (dict(pages=0), B.PA_ERR_INVALID),
    (dict(hq=0), B.PA_ERR_INVALID),
    (dict(d=64, qs=512), B.PA_ERR_UNSUPPORTED),
    (dict(P=48), B.PA_ERR_UNSUPPORTED),
    (dict(rot=8), B.PA_ERR_UNSUPPORTED),
    (dict(rot=40), B.PA_ERR_UNSUPPORTED),
    (dict(rot=144), B.PA_ERR_UNSUPPORTED),
])
def test_rope_refusals(lib, over, status):
    assert _caller(lib.pa_rope_append, ROPE)(**over) == status


TREE = dict(q=FAKE, k=FAKE, v=FAKE, ks=None, vs=None, kv=0, pt=FAKE, pts=16, cl=FAKE, cq=FAKE, mask=FAKE,
            words=1, bs=2, total=8, mql=4, hq=32, hkv=8, d=128, P=64, pages=100, msp=16, S=4, scale=0.1,
            ws=FAKE, wsb=1 << 30, out=FAKE, lse=None, stream=None, pdl=1)


@pytest.mark.parametrize("over,status", [
    (dict(bs=0), B.PA_OK),
    (dict(total=0), B.PA_OK),
    (dict(total=-1), B.PA_ERR_INVALID),
    (dict(mask=None), B.PA_ERR_INVALID),
    (dict(cq=None), B.PA_ERR_INVALID),
    (dict(out=None), B.PA_ERR_INVALID),
    (dict(out=FAKE + 4), B.PA_ERR_INVALID),
    (dict(mql=0), B.PA_ERR_INVALID),
    (dict(mql=65), B.PA_ERR_INVALID),              # two mask words needed
    (dict(mql=300, words=5), B.PA_ERR_UNSUPPORTED),
    (dict(ws=None), B.PA_ERR_INVALID),
    (dict(wsb=100), B.PA_ERR_INVALID),
    (dict(S=-1), B.PA_ERR_INVALID),
    (dict(scale=0.0), B.PA_ERR_INVALID), (dict(scale=-1.0), B.PA_ERR_INVALID),
    (dict(scale=math.nan), B.PA_ERR_INVALID), (dict(scale=math.inf), B.PA_ERR_INVALID),
    (dict(S=5000), B.PA_ERR_INVALID),
    (dict(hq=30), B.PA_ERR_INVALID),
    (dict(hq=256), B.PA_ERR_UNSUPPORTED),          # group 32
    (dict(hq=24), B.PA_ERR_UNSUPPORTED),           # group 3
    (dict(d=64), B.PA_ERR_UNSUPPORTED),
    (dict(P=8), B.PA_ERR_UNSUPPORTED),
    (dict(kv=1), B.PA_ERR_INVALID),
    (dict(pts=8), B.PA_ERR_INVALID),
    (dict(msp=1 << 24, pts=1 << 24), B.PA_ERR_UNSUPPORTED),  # positions past 2^29
    (dict(msp=1 << 22, pts=1 << 22, bs=1000), B.PA_ERR_UNSUPPORTED),  # chunks past 2^30
])
def test_tree_refusals(lib, over, status):
    assert _caller(lib.pa_tree_attention, TREE)(**over) == status


def test_tree_step_is_refused_before_anything_is_enqueued(lib):
    # (with no GPU an enqueued metadata kernel would come back as a CUDA error)
    def step(mql=4, words=1, total=8, q_mode=B.PA_Q_MODE_CUMSUM, qlens=FAKE, r2t=1024):
        return lib.pa_decode_step_tree(
            FAKE, FAKE, FAKE, 4, r2t, None, 0, 0, 16, FAKE, FAKE, FAKE, 16, None, 16, qlens, q_mode,
            0, FAKE, FAKE, words, FAKE, total, mql, FAKE, FAKE, None, None, 0, 2, 32, 8, 128, 64,
            100, 4, 0.1, FAKE, 1 << 30, FAKE, None, None, 1)
    assert step(mql=65) == B.PA_ERR_INVALID
    assert step(mql=300, words=5) == B.PA_ERR_UNSUPPORTED
    assert step(qlens=None) == B.PA_ERR_INVALID
    assert step(q_mode=7) == B.PA_ERR_INVALID
    assert step(r2t=15 * 64) == B.PA_ERR_INVALID
    assert step(total=0, r2t=15 * 64) == B.PA_ERR_INVALID


MASK = dict(parents=FAKE, cq=FAKE, bs=2, total=8, mql=4, mask=FAKE, words=1, stream=None, pdl=1)


@pytest.mark.parametrize("over,status", [
    (dict(bs=0), B.PA_OK), (dict(total=0), B.PA_OK), (dict(parents=None), B.PA_ERR_INVALID),
    (dict(mql=0), B.PA_ERR_INVALID), (dict(mql=70), B.PA_ERR_INVALID),
    (dict(mql=257, words=5), B.PA_ERR_UNSUPPORTED), (dict(mask=FAKE + 4), B.PA_ERR_INVALID),
])
def test_tree_mask_refusals(lib, over, status):
    assert _caller(lib.pa_build_tree_mask, MASK)(**over) == status


WEIGHTS = dict(q=FAKE, lse=FAKE, k=FAKE, ks=None, kv=0, pt=FAKE, pts=16, cl=FAKE, w=FAKE, bs=2, hq=32,
               hkv=8, d=128, P=64, pages=100, msp=16, scale=0.1, stream=None, pdl=1)


@pytest.mark.parametrize("over,status", [
    (dict(bs=0), B.PA_OK), (dict(q=None), B.PA_ERR_INVALID), (dict(lse=None), B.PA_ERR_INVALID),
    (dict(w=None), B.PA_ERR_INVALID), (dict(w=FAKE + 4), B.PA_ERR_INVALID),
    (dict(kv=1), B.PA_ERR_INVALID), (dict(hq=24), B.PA_ERR_UNSUPPORTED),
    (dict(d=64), B.PA_ERR_UNSUPPORTED), (dict(P=256), B.PA_ERR_UNSUPPORTED),
    (dict(msp=0), B.PA_ERR_INVALID),
    (dict(msp=(1 << 24) + 1, pts=1 << 25), B.PA_ERR_UNSUPPORTED),   # positions past 2^30
])
def test_weights_refusals(lib, over, status):
    assert _caller(lib.pa_accumulate_weights, WEIGHTS)(**over) == status


COMPACT = dict(pt=FAKE, pts=16, cl=FAKE, msp=16, kept=FAKE, heads=8, ks=100, counts=FAKE + 64, begin=None,
               max_kept=100, k=FAKE, v=FAKE, ksc=None, vsc=None, kv=0, w=None, dpt=FAKE, dpts=16, dmp=16,
               new=FAKE + 128, bs=2, hkv=8, d=128, P=64, pages=100, stream=None, pdl=1)


@pytest.mark.parametrize("over,status", [
    (dict(bs=0), B.PA_OK), (dict(kept=None), B.PA_ERR_INVALID), (dict(counts=None), B.PA_ERR_INVALID),
    (dict(heads=2), B.PA_ERR_INVALID), (dict(ks=50), B.PA_ERR_INVALID),
    (dict(max_kept=-1), B.PA_ERR_INVALID), (dict(new=FAKE), B.PA_ERR_INVALID),   # cache_seqlens
    (dict(new=FAKE + 64), B.PA_ERR_INVALID),                                        # counts
    (dict(dpts=17), B.PA_ERR_INVALID),                   # in place with another stride
    (dict(dpt=FAKE + 256, dmp=0), B.PA_ERR_INVALID), (dict(dpt=FAKE + 256, dmp=20), B.PA_ERR_INVALID),
    (dict(kv=1), B.PA_ERR_INVALID), (dict(P=20), B.PA_ERR_UNSUPPORTED), (dict(d=256), B.PA_ERR_UNSUPPORTED),
    (dict(begin=FAKE + 128), B.PA_ERR_INVALID),          # new_seqlens
    (dict(msp=(1 << 24) + 1, pts=1 << 25, dpts=1 << 25), B.PA_ERR_UNSUPPORTED),   # positions past 2^30
    (dict(max_kept=(1 << 30) + 1, ks=1 << 31), B.PA_ERR_UNSUPPORTED),
])
def test_compact_refusals(lib, over, status):
    assert _caller(lib.pa_compact_cache, COMPACT)(**over) == status


EVICT = dict(pt=FAKE, pts=16, cl=FAKE, msp=16, w=FAKE, k=FAKE, v=FAKE, ksc=None, vsc=None, kv=0, budget=100,
             first=4, recent=32, dpt=FAKE, dpts=16, dmp=16, kept=FAKE, new=FAKE + 64, bs=2, hkv=8, d=128,
             P=64, pages=100, stream=None, pdl=1)


@pytest.mark.parametrize("over,status", [
    (dict(bs=0), B.PA_OK), (dict(w=None), B.PA_ERR_INVALID), (dict(new=None), B.PA_ERR_INVALID),
    (dict(new=FAKE), B.PA_ERR_INVALID), (dict(budget=0), B.PA_ERR_INVALID),
    (dict(w=FAKE + 4), B.PA_ERR_INVALID),
    (dict(first=-1), B.PA_ERR_INVALID), (dict(recent=97), B.PA_ERR_INVALID),
    (dict(first=2**31 - 1, recent=2**31 - 1, budget=2**31 - 1), B.PA_ERR_INVALID),
    (dict(dpt=FAKE + 256, dmp=1), B.PA_ERR_INVALID),     # 100 rows do not fit 64
    (dict(P=8), B.PA_ERR_UNSUPPORTED),
    (dict(msp=(1 << 24) + 1, pts=1 << 25, dpts=1 << 25), B.PA_ERR_UNSUPPORTED),   # positions past 2^30
])
def test_evict_refusals(lib, over, status):
    assert _caller(lib.pa_evict, EVICT)(**over) == status


def test_rope_frequencies_follow_their_definitions():
    d, base, L = 128, 10000.0, 4096
    f = [base ** (-2 * i / d) for i in range(d // 2)]
    turns = [L * x / (2 * math.pi) for x in f]

    def close(got, want):
        assert got.dtype == torch.float64 and got.shape == (d // 2,)
        # pow, log and a handful of products in float64
        assert max(abs(a / b - 1) for a, b in zip(got.tolist(), want)) < 1e-12

    close(B.pa_rope_frequencies(d), f)
    close(B.pa_rope_frequencies(d, base, B.PA_ROPE_LINEAR, factor=4.0), [x / 4 for x in f])
    wide = base * 8 ** (d / (d - 2))
    got = B.pa_rope_frequencies(d, base, B.PA_ROPE_BASE, factor=8.0)
    close(got, [wide ** (-2 * i / d) for i in range(d // 2)])
    assert abs(got[-1].item() / (f[-1] / 8) - 1) < 1e-12   # the slowest pair, slowed 8 times
    got = B.pa_rope_frequencies(d, base, B.PA_ROPE_WAVELENGTH, factor=8.0, original_length=L,
                                low=1.0, high=4.0).tolist()
    for x, t, y in zip(f, turns, got):
        if t > 4:
            assert abs(y / x - 1) < 1e-12
        elif t < 1:
            assert abs(y / (x / 8) - 1) < 1e-12
        else:
            s = (t - 1) / 3
            assert abs(y / ((1 - s) * x / 8 + s * x) - 1) < 1e-12
    got = B.pa_rope_frequencies(d, base, B.PA_ROPE_BY_PARTS, factor=32.0, original_length=L,
                                low=1.0, high=32.0).tolist()
    assert all(b <= a for a, b in zip(got, got[1:]))
    for x, t, y in zip(f, turns, got):
        assert x / 32 * (1 - 1e-12) <= y <= x * (1 + 1e-12)
        if t > 40:
            assert abs(y / x - 1) < 1e-12
        if t < 0.8:
            assert abs(y / (x / 32) - 1) < 1e-12


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=128, base=1.0),
    dict(rotary_dim=128, base=math.nan), dict(rotary_dim=128, scaling=9),
    dict(rotary_dim=128, scaling=B.PA_ROPE_LINEAR, factor=0.0),
    dict(rotary_dim=2, scaling=B.PA_ROPE_BASE, factor=2.0),
    dict(rotary_dim=128, scaling=B.PA_ROPE_BY_PARTS, factor=2.0, original_length=0, low=1.0, high=32.0),
    dict(rotary_dim=128, scaling=B.PA_ROPE_WAVELENGTH, factor=2.0, original_length=10, low=4.0, high=4.0),
])
def test_rope_frequency_refusals(kw):
    with pytest.raises(B.PAError) as e:
        B.pa_rope_frequencies(**kw)
    assert e.value.status == B.PA_ERR_INVALID


def test_tree_splits_and_workspace():
    for (bs, mql, hq, hkv, P, msp), most in (((1, 8, 32, 8, 64, 16), 8), ((32, 32, 32, 8, 64, 128), 3),
                                             ((1, 1, 1, 1, 16, 1), 1), ((16, 64, 64, 8, 128, 128), 3),
                                             ((64, 256, 64, 8, 16, 1024), 2)):
        # no more pieces than chunks of 128 tokens; two or three once units outnumber the SMs
        assert 1 <= B.pa_choose_tree_splits(bs, mql, hq, hkv, P, msp, 152) <= most
    assert B.pa_choose_tree_splits(0, 8, 32, 8, 64, 16, 152) == 1
    assert B.pa_tree_workspace_bytes(0, 0, 0, 0, 0, 128, 64, 0) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    pool = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        B.pa_rope_append(q=x, k=x[:, :2], v=x[:, :2], positions=i, slots=i,
                         inv_freq=torch.ones(64, dtype=torch.float64), q_out=x, k_cache=pool, v_cache=pool)
    with pytest.raises(ValueError, match="shape"):
        B._shape(x, (2, 4, 128), "x")
    with pytest.raises(ValueError, match="contiguous"):
        B._token_rows(x.transpose(1, 2).contiguous().transpose(1, 2), 2, "q")
    with pytest.raises(ValueError, match="bf16"):
        B._token_rows(x.float(), 2, "q")
    assert B._token_rows(x[:, 2:4], 2, "k")[1:] == (1024, 2)   # a view of wider rows


# the same, with the rows' accumulated weights before the KV type
ROPE_WEIGHTS = {**{k: v for k, v in list(ROPE.items())[:22]}, "w": FAKE,
                **{k: v for k, v in list(ROPE.items())[22:]}}


@pytest.mark.parametrize("over,status", [
    (dict(tokens=0), B.PA_OK), (dict(tokens=-1), B.PA_ERR_INVALID), (dict(q=None), B.PA_ERR_INVALID),
    (dict(w=FAKE + 2), B.PA_ERR_INVALID),          # misaligned
    (dict(kv=1), B.PA_ERR_INVALID), (dict(P=48), B.PA_ERR_UNSUPPORTED), (dict(rot=8), B.PA_ERR_UNSUPPORTED),
])
def test_rope_with_weights_refusals(lib, over, status):
    assert list(ROPE_WEIGHTS)[21:24] == ["vsc", "w", "kv"]
    assert _caller(lib.pa_rope_append_weights, ROPE_WEIGHTS)(**over) == status


@pytest.mark.parametrize("scale", [math.nan, math.inf, -math.inf, 3e38])
def test_weights_refuse_a_scale_that_is_not_finite(lib, scale):
    """(3e38: not finite in base 2.)  Scales of 0 and below are a step's like any other."""
    assert _caller(lib.pa_accumulate_weights, WEIGHTS)(scale=scale) == B.PA_ERR_INVALID


def test_tree_refuses_a_scale_that_is_not_finite_in_base_2(lib):
    assert _caller(lib.pa_tree_attention, TREE)(scale=3e38) == B.PA_ERR_INVALID


def test_compact_and_evict_need_their_lists(lib):
    assert _caller(lib.pa_compact_cache, COMPACT)(kept=None, max_kept=1, ks=1) == B.PA_ERR_INVALID
    assert _caller(lib.pa_evict, EVICT)(kept=None) == B.PA_ERR_INVALID


@pytest.mark.parametrize("msp,splits", [((1 << 14) + 1, 1), ((1 << 14) + 1, 2), ((1 << 15) + 1, 3), (1 << 23, 512)])
def test_tree_refuses_pieces_past_2_to_20_tokens(lib, msp, splits):
    assert _caller(lib.pa_tree_attention, TREE)(msp=msp, pts=msp, S=splits, wsb=1 << 40) == B.PA_ERR_UNSUPPORTED


def test_tree_splits_of_long_contexts():
    # at least a piece for every 2^17 tokens and one more, from 2^18 tokens on
    for tokens in (1 << 19, 1 << 20, 1 << 24):
        assert B.pa_choose_tree_splits(64, 8, 32, 8, 64, tokens // 64, 152) >= (tokens >> 17) + 1
    assert B.pa_choose_tree_splits(64, 8, 32, 8, 64, 1 << 23, 152) == 4096
    assert B.pa_choose_tree_splits(64, 8, 32, 8, 64, (1 << 18) // 64, 152) <= 3


@pytest.mark.parametrize("d,base,length,factor", [(128, 10000.0, 4096, 32.0), (64, 500000.0, 8192, 8.0),
                                                  (16, 10000.0, 2048, 4.0)])
def test_rope_by_parts_ramp(d, base, length, factor):
    """Every pair of the ramp, from the header's formula."""
    pair = lambda turns: d * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))
    lo, hi = max(0, math.floor(pair(32.0))), min(d - 1, math.ceil(pair(1.0)))
    assert hi - lo >= 2
    got = B.pa_rope_frequencies(d, base, B.PA_ROPE_BY_PARTS, factor=factor, original_length=length, low=1.0,
                                high=32.0).tolist()
    for i, y in enumerate(got):
        f = base ** (-2 * i / d)
        r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        assert abs(y / (f * (1 - r) + f / factor * r) - 1) < 1e-12
