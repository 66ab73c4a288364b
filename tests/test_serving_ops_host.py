"""Host side of the block-scaled cache, the draft verification and the page operators: refusals
of the C entry points and of the binding, split counts (none of these calls reaches a GPU)."""

import ctypes
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


APPEND = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, pos=FAKE, freq=FAKE, rot=128, inter=0,
              amp=1.0, cu=FAKE, cl=FAKE, pt=FAKE, pts=16, msp=16, bs=2, total=5, mql=4, hq=8, hkv=2, d=128,
              qo=FAKE + 4096, qos=1024, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, kv=2, block=64, P=64,
              pages=10, stream=None, pdl=1)


@pytest.mark.parametrize("over,status", [
    (dict(bs=0), B.PA_OK), (dict(total=0), B.PA_OK), (dict(bs=-1), B.PA_ERR_INVALID),
    (dict(total=-1), B.PA_ERR_INVALID), (dict(cu=None), B.PA_ERR_INVALID),
    (dict(cl=None), B.PA_ERR_INVALID), (dict(pt=None), B.PA_ERR_INVALID),
    (dict(k=None), B.PA_ERR_INVALID), (dict(v=FAKE + 8), B.PA_ERR_INVALID),
    (dict(q=None), B.PA_ERR_INVALID), (dict(qo=None), B.PA_ERR_INVALID),
    (dict(pos=None), B.PA_ERR_INVALID), (dict(freq=None), B.PA_ERR_INVALID),
    (dict(ks=255), B.PA_ERR_INVALID), (dict(qs=1028), B.PA_ERR_INVALID),
    (dict(qo=FAKE, qos=2048), B.PA_ERR_INVALID),            # in place with another stride
    (dict(amp=math.nan), B.PA_ERR_INVALID), (dict(mql=0), B.PA_ERR_INVALID),
    (dict(kv=0), B.PA_ERR_INVALID), (dict(kv=1), B.PA_ERR_INVALID),
    (dict(ksc=None), B.PA_ERR_INVALID), (dict(vsc=FAKE + 2), B.PA_ERR_INVALID),
    (dict(P=32), B.PA_ERR_INVALID),                          # a block larger than a page
    (dict(block=8), B.PA_ERR_UNSUPPORTED), (dict(P=48), B.PA_ERR_UNSUPPORTED),
    (dict(P=256, block=128), B.PA_ERR_UNSUPPORTED), (dict(d=64), B.PA_ERR_UNSUPPORTED),
    (dict(rot=8), B.PA_ERR_UNSUPPORTED), (dict(rot=144), B.PA_ERR_UNSUPPORTED),
    (dict(rot=-16), B.PA_ERR_UNSUPPORTED), (dict(hq=-1), B.PA_ERR_INVALID),
    (dict(hkv=0), B.PA_ERR_INVALID), (dict(bs=65536), B.PA_ERR_INVALID),
    (dict(pts=8), B.PA_ERR_INVALID), (dict(msp=0), B.PA_ERR_INVALID), (dict(pages=0), B.PA_ERR_INVALID),
    (dict(msp=1 << 24, pts=1 << 24), B.PA_ERR_UNSUPPORTED),  # positions past 2^29
])
def test_append_refusals(lib, over, status):
    assert _caller(lib.pa_rope_append_blocks, APPEND)(**over) == status


ATTEND = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, kv=2, block=64, pt=FAKE, pts=16, cl=FAKE, cu=FAKE,
              bs=2, total=8, mql=4, hq=32, hkv=8, d=128, P=64, pages=100, msp=16, S=4, scale=0.1, ws=FAKE,
              wsb=1 << 30, out=FAKE, lse=None, stream=None, pdl=1)


@pytest.mark.parametrize("over,status", [
    (dict(bs=0), B.PA_OK), (dict(total=0), B.PA_OK), (dict(total=-1), B.PA_ERR_INVALID),
    (dict(q=None), B.PA_ERR_INVALID), (dict(q=FAKE + 8), B.PA_ERR_INVALID),
    (dict(out=None), B.PA_ERR_INVALID), (dict(out=FAKE + 4), B.PA_ERR_INVALID),
    (dict(lse=FAKE + 1), B.PA_ERR_INVALID), (dict(ks=None), B.PA_ERR_INVALID),
    (dict(vs=None), B.PA_ERR_INVALID), (dict(kv=0), B.PA_ERR_INVALID), (dict(kv=3), B.PA_ERR_INVALID),
    (dict(cu=None), B.PA_ERR_INVALID),                       # one query a request: total = bs
    (dict(mql=0), B.PA_ERR_INVALID), (dict(S=-1), B.PA_ERR_INVALID), (dict(S=4097), B.PA_ERR_INVALID),
    (dict(ws=None), B.PA_ERR_INVALID), (dict(wsb=100), B.PA_ERR_INVALID), (dict(ws=FAKE + 8), B.PA_ERR_INVALID),
    (dict(scale=math.inf), B.PA_ERR_INVALID), (dict(scale=math.nan), B.PA_ERR_INVALID),
    (dict(hq=30), B.PA_ERR_INVALID), (dict(hq=0), B.PA_ERR_INVALID),
    (dict(hq=264), B.PA_ERR_UNSUPPORTED),                    # 33 heads to a kv head
    (dict(mql=70000), B.PA_ERR_UNSUPPORTED), (dict(d=256), B.PA_ERR_UNSUPPORTED),
    (dict(block=128), B.PA_ERR_INVALID), (dict(P=8, block=8), B.PA_ERR_UNSUPPORTED),
    (dict(pts=8), B.PA_ERR_INVALID), (dict(msp=1 << 24, pts=1 << 24), B.PA_ERR_UNSUPPORTED),
    (dict(msp=1 << 22, pts=1 << 22, bs=1000), B.PA_ERR_UNSUPPORTED),   # chunks past 2^30
])
def test_attention_refusals(lib, over, status):
    assert _caller(lib.pa_block_attention, ATTEND)(**over) == status


def test_step_is_refused_before_anything_is_enqueued(lib):
    # (with no GPU an enqueued metadata kernel would come back as a CUDA error)
    def step(total=8, mql=4, cu=FAKE, q_mode=B.PA_Q_MODE_CUMSUM, qlens=FAKE, r2t=1024, kv=2, block=64):
        return lib.pa_decode_step_block(
            FAKE, FAKE, FAKE, 4, r2t, None, 0, 0, 16, FAKE, FAKE, FAKE, 16, None, 16, qlens, q_mode, 0, cu,
            FAKE, total, mql, FAKE, FAKE, FAKE, FAKE, kv, block, 2, 32, 8, 128, 64, 100, 4, 0.1, FAKE,
            1 << 30, FAKE, None, None, 1)
    assert step(kv=0) == B.PA_ERR_INVALID
    assert step(block=8) == B.PA_ERR_UNSUPPORTED
    assert step(mql=0) == B.PA_ERR_INVALID
    assert step(qlens=None) == B.PA_ERR_INVALID
    assert step(q_mode=7) == B.PA_ERR_INVALID
    assert step(r2t=15 * 64) == B.PA_ERR_INVALID
    assert step(cu=None, q_mode=B.PA_Q_MODE_NONE, qlens=None) == B.PA_ERR_INVALID   # total is not bs
    assert step(total=0, r2t=15 * 64) == B.PA_ERR_INVALID


def test_block_splits_and_workspace():
    for args, most in (((1, 1, 32, 8, 64, 16), 8), ((32, 1, 32, 8, 64, 128), 5), ((1, 1, 1, 1, 16, 1), 1),
                       ((64, 1, 64, 8, 64, 256), 3), ((1, 1, 32, 8, 64, 128), 64)):
        assert 1 <= B.pa_choose_block_splits(*args, 152) <= most
    assert B.pa_choose_block_splits(0, 1, 32, 8, 64, 16, 152) == 1
    assert B.pa_choose_block_splits(1, 1, 33, 1, 64, 16, 152) == 1
    assert B.pa_choose_block_splits(1, 1, 8, 1, 16, 1 << 25, 152) <= 4096
    assert B.pa_block_workspace_bytes(0, 0, 0, 0, 0, 128, 64, 0) == 0


VERIFY = dict(p=FAKE, ps=1000, q=FAKE, qs=1000, vocab=1000, tok=FAKE, par=FAKE, cu=FAKE, cl=FAKE, u=FAKE,
              fu=FAKE, bs=2, total=8, mql=4, kept=FAKE, kepts=4, counts=FAKE + 64, begin=FAKE + 128, nxt=FAKE,
              stream=None, pdl=1)


@pytest.mark.parametrize("over,status", [
    (dict(bs=0), B.PA_OK), (dict(bs=-1), B.PA_ERR_INVALID), (dict(total=-1), B.PA_ERR_INVALID),
    (dict(p=None), B.PA_ERR_INVALID), (dict(tok=None), B.PA_ERR_INVALID), (dict(u=None), B.PA_ERR_INVALID),
    (dict(fu=None), B.PA_ERR_INVALID), (dict(kept=None), B.PA_ERR_INVALID),
    (dict(counts=None), B.PA_ERR_INVALID), (dict(nxt=None), B.PA_ERR_INVALID),
    (dict(p=FAKE + 2), B.PA_ERR_INVALID), (dict(tok=FAKE + 4), B.PA_ERR_INVALID),
    (dict(ps=999), B.PA_ERR_INVALID), (dict(qs=999), B.PA_ERR_INVALID), (dict(vocab=0), B.PA_ERR_INVALID),
    (dict(mql=0), B.PA_ERR_INVALID), (dict(kepts=3), B.PA_ERR_INVALID), (dict(bs=65536), B.PA_ERR_INVALID),
    (dict(counts=FAKE), B.PA_ERR_INVALID), (dict(begin=FAKE), B.PA_ERR_INVALID),   # cache_seqlens
    (dict(mql=257, kepts=300), B.PA_ERR_UNSUPPORTED),
    (dict(vocab=(1 << 20) + 1, ps=1 << 21, qs=1 << 21), B.PA_ERR_UNSUPPORTED),
])
def test_verify_refusals(lib, over, status):
    assert _caller(lib.pa_verify_drafts, VERIFY)(**over) == status


def pools(*pairs):
    array = (B._PagePool * max(len(pairs), 1))()
    for i, (base, size) in enumerate(pairs):
        array[i].base, array[i].page_bytes = base, size
    return array


GOOD = pools((FAKE, 4096), (FAKE, 4))
COPY = dict(src=GOOD, dst=None, n=2, ns=10, nd=10, sp=FAKE, dp=FAKE, count=3, stream=None, pdl=1)


@pytest.mark.parametrize("over,status", [
    (dict(count=0), B.PA_OK), (dict(n=0, src=None), B.PA_OK), (dict(count=-1), B.PA_ERR_INVALID),
    (dict(src=None), B.PA_ERR_INVALID), (dict(n=-1), B.PA_ERR_INVALID), (dict(sp=None), B.PA_ERR_INVALID),
    (dict(dp=FAKE + 2), B.PA_ERR_INVALID), (dict(ns=0), B.PA_ERR_INVALID), (dict(nd=0), B.PA_ERR_INVALID),
    (dict(src=pools((None, 4096), (FAKE, 4))), B.PA_ERR_INVALID),
    (dict(src=pools((FAKE + 2, 4096), (FAKE, 4))), B.PA_ERR_INVALID),
    (dict(src=pools((FAKE, 4098), (FAKE, 4))), B.PA_ERR_INVALID),
    (dict(src=pools((FAKE, 0), (FAKE, 4))), B.PA_ERR_INVALID),
    (dict(dst=pools((FAKE, 4096), (FAKE, 8))), B.PA_ERR_INVALID),   # pages of another size
])
def test_page_copy_refusals(lib, over, status):
    assert _caller(lib.pa_pages_copy, COPY)(**over) == status


TABLE = dict(t=FAKE, rows=10, stride=1024, refs=FAKE, pages=100, P=64, msp=16)
LISTS = {"pa_pages_fork": dict(r=FAKE, c=FAKE, lens=FAKE, count=3, pools=GOOD, n=2, out=FAKE + 64, ws=FAKE,
                               wsb=1 << 20, stream=None, pdl=1),
         "pa_pages_extend": dict(r=FAKE, lens=FAKE, new=FAKE + 32, count=3, out=FAKE + 64, ws=FAKE, wsb=1 << 20,
                                 stream=None, pdl=1),
         "pa_pages_free": dict(r=FAKE, lens=FAKE, keep=None, count=3, stream=None, pdl=1),
         "pa_pages_compact": dict(r=FAKE, lens=FAKE, count=3, pools=GOOD, n=2, map=FAKE, live=FAKE, ws=FAKE,
                                  wsb=1 << 20, stream=None, pdl=1)}


@pytest.mark.parametrize("name", sorted(LISTS))
@pytest.mark.parametrize("over,status", [
    (dict(count=-1), B.PA_ERR_INVALID), (dict(t=None), B.PA_ERR_INVALID), (dict(refs=None), B.PA_ERR_INVALID),
    (dict(r=None), B.PA_ERR_INVALID), (dict(lens=None), B.PA_ERR_INVALID), (dict(t=FAKE + 2), B.PA_ERR_INVALID),
    (dict(r=FAKE + 4), B.PA_ERR_INVALID), (dict(rows=0), B.PA_ERR_INVALID), (dict(pages=0), B.PA_ERR_INVALID),
    (dict(P=0), B.PA_ERR_INVALID), (dict(msp=0), B.PA_ERR_INVALID),
    (dict(stride=15 * 64), B.PA_ERR_INVALID),                # the last page would not start in a row
    (dict(pages=1 << 20, P=1 << 11, msp=1), B.PA_ERR_INVALID),       # slots past int32
    (dict(pages=(1 << 20) + 1, P=16), B.PA_ERR_UNSUPPORTED), (dict(count=65536), B.PA_ERR_UNSUPPORTED),
    (dict(msp=(1 << 23) + 1, stride=1 << 30), B.PA_ERR_UNSUPPORTED),
])
def test_page_table_refusals(lib, name, over, status):
    assert _caller(getattr(lib, name), TABLE | LISTS[name])(**over) == status


@pytest.mark.parametrize("name,over,status", [
    ("pa_pages_fork", dict(count=0), B.PA_OK), ("pa_pages_extend", dict(count=0), B.PA_OK),
    ("pa_pages_free", dict(count=0), B.PA_OK),
    ("pa_pages_fork", dict(c=None), B.PA_ERR_INVALID), ("pa_pages_fork", dict(out=None), B.PA_ERR_INVALID),
    ("pa_pages_fork", dict(out=FAKE), B.PA_ERR_INVALID),     # lens
    ("pa_pages_fork", dict(ws=None), B.PA_ERR_INVALID), ("pa_pages_fork", dict(wsb=100), B.PA_ERR_INVALID),
    ("pa_pages_fork", dict(pools=pools((FAKE, 3)), n=1), B.PA_ERR_INVALID),
    ("pa_pages_extend", dict(new=None), B.PA_ERR_INVALID), ("pa_pages_extend", dict(out=FAKE), B.PA_ERR_INVALID),
    ("pa_pages_extend", dict(out=FAKE + 32), B.PA_ERR_INVALID), ("pa_pages_extend", dict(ws=FAKE + 8), B.PA_ERR_INVALID),
    ("pa_pages_compact", dict(map=None), B.PA_ERR_INVALID), ("pa_pages_compact", dict(live=None), B.PA_ERR_INVALID),
    ("pa_pages_compact", dict(wsb=0), B.PA_ERR_INVALID),
    ("pa_pages_compact", dict(pools=None), B.PA_ERR_INVALID),
    ("pa_pages_compact", dict(r=None, lens=None, count=0, map=None), B.PA_ERR_INVALID),
])
def test_page_list_refusals(lib, name, over, status):
    assert _caller(getattr(lib, name), TABLE | LISTS[name])(**over) == status


def test_pages_workspace():
    assert B.pa_pages_workspace_bytes(100, 3) == 256 + 3 * 512
    assert B.pa_pages_workspace_bytes(10, 300) == 256 + 3 * 1280
    assert B.pa_pages_workspace_bytes(-1, 3) == 0


def test_the_calls_that_take_other_pools_refuse_e4m3(lib):
    """bf16 and int8 calls do not read a block-scaled pool by mistake."""
    assert lib.pa_decode_splitk(FAKE, FAKE, FAKE, FAKE, FAKE, B.PA_KV_E4M3, FAKE, 16, FAKE, 2, 32, 8, 128, 64, 100,
                                16, 4, 0.1, FAKE, FAKE, FAKE, None, 1) == B.PA_ERR_INVALID
    pool = torch.zeros((4, 2, 16, 128), dtype=torch.float8_e4m3fn)
    with pytest.raises((ValueError, TypeError)):
        B._kv_args(pool, pool, None, None)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    pool = torch.zeros((4, 2, 16, 128), dtype=torch.float8_e4m3fn)
    scale = torch.zeros((4, 2, 1))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        B.pa_block_attention(q=torch.zeros((1, 4, 128), dtype=torch.bfloat16), k_cache=pool, v_cache=pool,
                             k_scale=scale, v_scale=scale, page_table=torch.zeros((1, 1), dtype=torch.int32),
                             cache_seqlens=torch.zeros(1, dtype=torch.int32), max_seq_pages=1, sm_scale=0.1,
                             out=torch.zeros((1, 4, 128), dtype=torch.bfloat16))
    assert B._block_pools(pool, pool, scale, scale) == (16, (4, 2, 16, 128))
    with pytest.raises(ValueError, match="e4m3"):
        B._block_pools(pool.to(torch.bfloat16), pool, scale, scale)
    with pytest.raises(ValueError, match="v_scale"):
        B._block_pools(pool, pool, scale, scale[:3])
    with pytest.raises(ValueError, match="k_scale"):
        B._block_pools(pool, pool, torch.zeros((4, 2, 3)), scale)
    with pytest.raises(ValueError, match="pages"):
        B._page_pools([torch.zeros((3, 4))], 4, "pools")
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        B._page_pools([torch.zeros((4, 4))], 4, "pools")
    with pytest.raises(ValueError, match="one query per request"):
        B._block_rows(torch.zeros((3, 4, 128)), None, torch.zeros(2), 1, torch.zeros((3, 4, 128)), None, 128)


def test_prepared_calls_keep_their_pools_alive():
    array = (ctypes.c_int64 * 2)(1, 2)
    x, y = torch.zeros(1), torch.zeros(2)
    call = B.PreparedCall("pa_choose_splits", (1, 1, 1, 16, 0, 152), keep=(x, [y], array, None, 3))
    assert any(k is array for k in call._keep) and any(k is y for k in call._keep) and len(call._keep) == 3


@pytest.mark.parametrize("name,defaults,pointers", [
    ("pa_rope_append_blocks", APPEND, ("cu", "cl", "pt")),
    ("pa_block_attention", ATTEND, ("cu", "cl", "pt")),
    ("pa_verify_drafts", VERIFY, ("par", "cu", "cl", "u", "fu", "kept", "counts", "begin")),
    ("pa_pages_fork", TABLE | LISTS["pa_pages_fork"], ("lens", "refs", "out")),
    ("pa_pages_extend", TABLE | LISTS["pa_pages_extend"], ("lens", "new", "out")),
    ("pa_pages_free", TABLE | LISTS["pa_pages_free"], ("lens", "keep")),
    ("pa_pages_compact", TABLE | LISTS["pa_pages_compact"], ("lens", "map", "live")),
])
def test_index_arrays_off_their_alignment_are_refused(lib, name, defaults, pointers):
    for pointer in pointers:
        assert _caller(getattr(lib, name), defaults)(**{pointer: FAKE + 256 + 2}) == B.PA_ERR_INVALID, pointer


def test_tables_that_are_columns_of_wider_ones():
    """Slots are written up to the row's stride, so a last page must not reach past the columns of
    a view.  (A host tensor is refused, too, but after the table's shape.)"""
    big = torch.zeros((4, 256), dtype=torch.int32)
    refs, one = torch.zeros(9, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    lens = torch.zeros(1, dtype=torch.int32)
    for table, pages in ((big[:, 200:256], 1), (big[:, :200], 4), (big[:, 64:129], 2), (big[3:, 250:], 2),
                         (big, 5)):
        with pytest.raises(ValueError, match="room for fewer"):
            B._slot_table(table, refs, 64, pages, one, lens)
    for table, pages in ((big[:, 64:192], 2), (big[:, :200], 3), (big, 4), (big[:, :200].contiguous(), 4),
                         (big[3:, 200:256], 1)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            B._slot_table(table, refs, 64, pages, one, lens)


@pytest.mark.parametrize("msp,P,status", [(1021, 128, B.PA_ERR_INVALID), (1022, 128, B.PA_ERR_UNSUPPORTED),
                                          (2 * 1021, 64, B.PA_ERR_INVALID), (2 * 1021 + 1, 64, B.PA_ERR_UNSUPPORTED)])
def test_the_largest_batch_of_chunks(lib, msp, P, status):
    """2^20 tiles (1024 requests, 1024 kv heads) of 1021 chunks of 128 tokens, and two more a tile for what
    it costs beside them, are the most.  (Invalid: past that check, but without a workspace.)"""
    assert _caller(lib.pa_block_attention, ATTEND)(bs=1024, total=1024, mql=1, hq=1024, hkv=1024, P=P, msp=msp,
                                                   pts=1 << 12, ws=None) == status
