"""Failure detection of the tree attention without a GPU fault: with loads held back (a hook of
the instrumented build) its waits run out, the call returns and reports it, nothing is written of
rows that one block has, and the context, and the next call, are as if nothing had been."""

import time

import pytest
import torch

import cache_reference as R
from paged_kv_decode_metadata_gb300 import binding as B
from paged_kv_decode_metadata_gb300 import build
from test_gpu_cache_ops import SCALE, Cache, Tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ts():
    build.build(instrumented=True)
    lib = B.load_instrumented()
    B.pa_read_error_flags(reset=True, lib=lib)
    yield lib
    lib.pa_set_test_hold_loads(0)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("nodes,splits", [(5, 1), (60, 1), (5, 3)])
def test_tree_wait_limit_reports_and_returns(ts, kv, nodes, splits):
    """One tile of rows and two; whole contexts and cut ones."""
    c = Cache([700, 1100, 600], 2, 64, kv, 61)
    t = Tree(c, [nodes] * 3, 8, 62)
    out = torch.full((t.total, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((t.total, 8), 7.0, device="cuda")
    call = B.prepare_tree_attention(
        lib=ts, q=t.q.cuda(), k_cache=c.d_k, v_cache=c.d_v, k_scale=c.d_ks, v_scale=c.d_vs, page_table=c.d_table,
        cache_seqlens=c.d_n, cu_seqlens_q=t.cu.cuda(), tree_mask=R.mask_tensor(t.masks, t.words).cuda(),
        max_q_len=nodes, max_seq_pages=c.msp, num_splits=splits, sm_scale=SCALE, out=out, lse=lse,
        workspace=torch.full((B.pa_workspace_bytes(t.total, 8, 128, splits),), 255, dtype=torch.uint8, device="cuda"))
    assert ts.pa_set_test_hold_loads(1) == B.PA_OK
    try:
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
    t.check(out, lse)
