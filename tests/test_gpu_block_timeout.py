"""Failure detection of the block attention without a GPU fault: with loads held back (a hook of
the instrumented build) its waits run out, the call returns and reports it, nothing is written of
whole rows, and the context, and the next call, are as if nothing had been."""

import time

import pytest
import torch

import block_reference as R
from paged_kv_decode_metadata_gb300 import binding as B
from paged_kv_decode_metadata_gb300 import build
from test_gpu_block_cache import SCALE, BlockCache, blank, check, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ts():
    build.build(instrumented=True)
    lib = B.load_instrumented()
    B.pa_read_error_flags(reset=True, lib=lib)
    yield lib
    lib.pa_set_test_hold_loads(0)


@pytest.mark.parametrize("hq,q_len,splits", [(8, 1, 1), (16, 3, 1), (16, 8, 1), (8, 1, 4), (16, 8, 3)])
def test_wait_limit_reports_and_returns(ts, hq, q_len, splits):
    """8, 16 (6 x 3) and 32 columns; whole contexts and cut ones."""
    c = BlockCache([700, 1100, 600], 2, 64, 32, 61)
    q = torch.randn((3 * q_len, hq, 128), generator=c.g).to(torch.bfloat16)
    out, lse = blank(3 * q_len, hq)
    call = B.prepare_block_attention(
        lib=ts, q=q.cuda(), k_cache=c.d_k, v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs, page_table=c.d_table,
        cache_seqlens=c.d_n, cu_seqlens_q=rows_of([q_len] * 3).cuda(), max_q_len=q_len, max_seq_pages=c.msp,
        num_splits=splits, sm_scale=SCALE, out=out, lse=lse,
        workspace=torch.full((B.pa_workspace_bytes(3 * q_len, hq, 128, splits),), 255, dtype=torch.uint8, device="cuda"))
    assert ts.pa_set_test_hold_loads(1) == B.PA_OK
    try:
        # (the hook is read when the call is made)
        start = time.perf_counter()
        call()
        torch.cuda.synchronize()
        waited = time.perf_counter() - start
    finally:
        ts.pa_set_test_hold_loads(0)
    assert B.pa_read_error_flags(reset=True, lib=ts) & B.DEVERR_WAIT_TIMEOUT
    assert 1.0 < waited < 60.0, waited                   # one wait limit, then a bounded drain
    if splits == 1:
        assert bool((out == 7.0).all()) and bool((lse == 7.0).all())
    for _ in range(3):                                   # the hook off: the right answer
        call()
    torch.cuda.synchronize()
    assert B.pa_read_error_flags(reset=True, lib=ts) == 0
    check(out, lse, R.attention(q, c.k, c.v, c.ks, c.vs, c.table, c.n, [q_len] * 3, SCALE))
