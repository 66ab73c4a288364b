"""A run of the serving operators together, as a loop uses them: pages handed out, a prompt and
drafts appended to a block-scaled cache, the step over it, the drafts verified, the rejected ones'
pages given back; requests forked, packed to the front of the pools, and the step captured."""

import pytest
import torch

import block_reference as R
import verify_reference as V
from paged_kv_decode_metadata_gb300 import binding as B
from paged_kv_decode_metadata_gb300 import build
from test_gpu_block_cache import SCALE, check, same

pytestmark = pytest.mark.gpu

HQ, HKV, PAGE, BLOCK, ROWS, MSP, PAGES, VOCAB = 8, 2, 32, 16, 6, 8, 30, 517


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    B.load()
    B.pa_read_error_flags(reset=True)
    yield
    assert B.pa_read_error_flags(reset=True) == 0


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype).cuda()


class Server:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.table = torch.full((ROWS, MSP * PAGE), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        shape = (PAGES, HKV, PAGE, 128)
        self.k, self.v = (torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                          for _ in "kv")
        self.ks, self.vs = (torch.full((PAGES, HKV, PAGE // BLOCK), float("nan"), device="cuda") for _ in "kv")
        self.inv = B.pa_rope_frequencies(128).cuda()
        self.lens = [0] * ROWS
        self.truth = [[None, None] for _ in range(ROWS)]     # float64 keys (turned) and values
        self.ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")

    @property
    def pools(self):
        return [self.k, self.v, self.ks, self.vs]

    def paged(self, lens):
        return dict(req_to_token=self.table, page_refs=self.refs, page_size=PAGE, max_seq_pages=MSP, lens=ints(lens))

    def extend(self, rows, new):
        granted = torch.zeros(len(rows), dtype=torch.int32, device="cuda")
        B.pa_pages_extend(rows=ints(rows, torch.int64), new_lens=ints(new), granted=granted, workspace=self.ws,
                          **self.paged([self.lens[r] for r in rows]))
        assert granted.tolist() == new

    def meta(self, rows, lens, counts):
        bs = len(rows)
        m = dict(req_pool_indices=ints(rows, torch.int64), seq_lens=ints(lens, torch.int64), req_to_token=self.table,
                 cache_seqlens=torch.zeros(bs, dtype=torch.int32, device="cuda"),
                 cu_seqlens_k=torch.zeros(bs + 1, dtype=torch.int32, device="cuda"),
                 page_table=torch.zeros((bs, MSP), dtype=torch.int32, device="cuda"))
        cu = torch.zeros(bs + 1, dtype=torch.int32, device="cuda")
        B.pa_build_metadata_full(**m, seqlen_offset=0, max_seq_pages=MSP, page_size=PAGE, cu_seqlens_q=cu,
                                 qlens=ints(counts, torch.int64), q_mode=B.PA_Q_MODE_CUMSUM)
        return m, cu

    def inputs(self, tokens):
        return torch.randn((tokens, HQ + 2 * HKV, 128), generator=self.g).to(torch.bfloat16)

    def append(self, rows, lens, counts, wide, m, cu):
        """The newest `counts` tokens of every row; returns the turned queries."""
        d = wide.cuda()
        q, k, v = d.split([HQ, HKV, HKV], dim=1)
        positions = torch.cat([torch.arange(n - c, n) for n, c in zip(lens, counts)])
        q_out = torch.empty((d.shape[0], HQ, 128), dtype=torch.bfloat16, device="cuda")
        B.pa_rope_append_blocks(q=q, q_out=q_out, k=k, v=v, positions=positions.cuda(), inv_freq=self.inv,
                                cu_seqlens_q=cu, cache_seqlens=m["cache_seqlens"], page_table=m["page_table"],
                                max_seq_pages=MSP, k_cache=self.k, v_cache=self.v, k_scale=self.ks, v_scale=self.vs)
        _, k, v = wide.split([HQ, HKV, HKV], dim=1)
        k = R.rope(k, positions, self.inv.cpu(), False, 1.0)
        at = 0
        for r, n, c in zip(rows, lens, counts):
            for i, x in enumerate((k, v.double())):
                old = self.truth[r][i]
                new = x[at:at + c]
                self.truth[r][i] = new if old is None else torch.cat((old[:n - c], new))
            at += c
        return q_out

    def step(self, q, m, cu, counts, lens, **kw):
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], device="cuda")
        B.pa_decode_step_block(**m, seqlen_offset=0, max_seq_pages=MSP, q=q, k_cache=self.k, v_cache=self.v,
                               k_scale=self.ks, v_scale=self.vs, sm_scale=SCALE, out=out, lse=lse, cu_seqlens_q=cu,
                               max_q_len=max(counts), qlens=ints(counts, torch.int64), q_mode=B.PA_Q_MODE_CUMSUM,
                               workspace=self.ws, **kw)
        return out, lse

    def check_step(self, out, lse, q, m, counts, lens):
        torch.cuda.synchronize()
        check(out, lse, R.attention(q.cpu(), self.k.cpu(), self.v.cpu(), self.ks.cpu(), self.vs.cpu(),
                                    m["page_table"].cpu(), lens, counts, SCALE))

    def check_rows(self, row, n):
        """What is cached is what was appended, to a code's rounding: half a step of e4m3 (2^-4 of
        the value), or of its smallest codes, whatever the scale has grown by (doubled for that)."""
        table = (self.table[row].cpu()[::PAGE] // PAGE).to(torch.int32)
        for i, (codes, scale) in enumerate(((self.k, self.ks), (self.v, self.vs))):
            for h in range(HKV):
                got = R.rows(codes.cpu(), scale.cpu(), table, n, h)
                want = self.truth[row][i][:n, h]
                step = scale.cpu().double()[table.long()[torch.arange(n) // PAGE], h,
                                            torch.arange(n) % PAGE // BLOCK][:, None]
                assert ((got - want).abs() <= 2.0 ** -4 * want.abs() + step * 2.0 ** -9).all()


def test_loop():
    s = Server(1)
    rows, s_lens = [1, 4], [37, 70]
    s.extend(rows, s_lens)
    m, cu = s.meta(rows, s_lens, s_lens)
    q = s.append(rows, s_lens, s_lens, s.inputs(sum(s_lens)), m, cu)
    out, lse = s.step(q, m, cu, s_lens, s_lens)          # the prompt itself, causally
    s.check_step(out, lse, q, m, s_lens, s_lens)
    for r, n in zip(rows, s_lens):
        s.lens[r] = n
    for turn in range(6):
        counts = [4, 1 + turn % 3]                        # the last token and its draft
        lens = [s.lens[r] + c for r, c in zip(rows, counts)]
        s.extend(rows, lens)
        m, cu = s.meta(rows, lens, counts)
        q = s.append(rows, lens, counts, s.inputs(sum(counts)), m, cu)
        out, lse = s.step(q, m, cu, counts, lens)
        s.check_step(out, lse, q, m, counts, lens)
        # verification by the probabilities of a made-up head
        target = torch.softmax(torch.randn((sum(counts), VOCAB), generator=s.g), -1)
        draft = torch.softmax(target.log() + 0.3 * torch.randn(target.shape, generator=s.g), -1)
        drawn = torch.multinomial(draft, 1, generator=s.g)[:, 0]
        tokens = torch.cat([torch.cat((torch.tensor([0]), drawn[a:a + c - 1])) for a, c in ((0, 4), (4, counts[1]))])
        u, fu = torch.rand(sum(counts), generator=s.g), torch.rand(2, generator=s.g)
        kept = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
        got, begin = (torch.zeros(2, dtype=torch.int32, device="cuda") for _ in "cb")
        nxt = torch.zeros(2, dtype=torch.int64, device="cuda")
        B.pa_verify_drafts(target_probs=target.cuda(), draft_probs=draft.cuda(), tokens=tokens.cuda(), cu_seqlens_q=cu,
                           cache_seqlens=m["cache_seqlens"], uniforms=u.cuda(), final_uniforms=fu.cuda(), max_q_len=4,
                           kept=kept, counts=got, begin=begin, next_tokens=nxt)
        new = (begin + got).tolist()
        at = 0
        for b, c in enumerate(counts):
            path, token = V.verify(target[at:at + c].numpy(), draft[at:at + c].numpy(), tokens[at:at + c].tolist(),
                                   [i - 1 for i in range(c)], u[at:at + c].tolist(), float(fu[b]))
            assert int(got[b]) == len(path) and int(nxt[b]) == token
            at += c
        # the rejected tokens' pages given back
        B.pa_pages_free(rows=ints(rows, torch.int64), keep_lens=ints(new), **s.paged(lens))
        for r, n in zip(rows, new):
            s.lens[r] = n
            s.check_rows(r, n)
    assert int(s.refs.sum()) == sum(-(-s.lens[r] // PAGE) for r in rows)

    # ----- forks: what a child sees is what its parent saw, and neither disturbs the other ------
    lens = [s.lens[1], s.lens[1], s.lens[4]]
    child = torch.zeros(3, dtype=torch.int32, device="cuda")
    B.pa_pages_fork(parents=ints([1, 1, 4], torch.int64), children=ints([0, 2, 5], torch.int64), pools=s.pools,
                    child_lens=child, workspace=s.ws, **s.paged(lens))
    assert child.tolist() == lens
    for r, p in ((0, 1), (2, 1), (5, 4)):
        s.lens[r], s.truth[r] = s.lens[p], list(s.truth[p])
    every = [1, 4, 0, 2, 5]
    now = [s.lens[r] for r in every]
    q = torch.randn((2, HQ, 128), generator=s.g).to(torch.bfloat16).cuda()[[0, 1, 0, 0, 1]].contiguous()
    m, cu = s.meta(every, now, [1] * 5)
    out, lse = s.step(q, m, cu, [1] * 5, now)
    s.check_step(out, lse, q, m, [1] * 5, now)
    for a, b in ((0, 2), (0, 3), (1, 4)):
        assert same(out[a], out[b]) and same(lse[a], lse[b])
    grown = [n + 1 for n in now]
    s.extend(every, grown)
    m, cu = s.meta(every, grown, [1] * 5)
    q = s.append(every, grown, [1] * 5, s.inputs(5), m, cu)
    for r, n in zip(every, grown):
        s.lens[r] = n
        s.check_rows(r, n)
    before = s.step(q, m, cu, [1] * 5, grown)
    s.check_step(*before, q, m, [1] * 5, grown)

    # ----- one parent ends; the others' pages move to the front, and nothing else changes ---------
    B.pa_pages_free(rows=ints([1], torch.int64), **s.paged([s.lens[1]]))
    left = [4, 0, 2, 5]
    page_map = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.pa_pages_compact(rows=ints(left, torch.int64), pools=s.pools, page_map=page_map, num_live=live, workspace=s.ws,
                       **s.paged([s.lens[r] for r in left]))
    assert int(live) == int((s.refs > 0).sum()) and bool((s.refs[:int(live)] > 0).all())
    m, cu = s.meta(left, grown[1:], [1] * 4)
    after = s.step(q[1:].contiguous(), m, cu, [1] * 4, grown[1:])
    torch.cuda.synchronize()
    s.check_step(*after, q[1:].contiguous(), m, [1] * 4, grown[1:])
    B.pa_pages_free(rows=ints(left, torch.int64), **s.paged([s.lens[r] for r in left]))
    assert int(s.refs.sum()) == 0


def test_captured_step_matches_eager():
    """Append, step and verification in one graph, replayed on new inputs."""
    s = Server(2)
    rows, lens, counts = [0, 3], [50, 90], [3, 3]
    s.extend(rows, [96, 128])
    m, cu = s.meta(rows, lens, lens)
    s.append(rows, lens, lens, s.inputs(sum(lens)), m, cu)
    torch.cuda.synchronize()
    d = s.inputs(6).cuda()
    q, k, v = d.split([HQ, HKV, HKV], dim=1)
    q_out = torch.empty((6, HQ, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q_out), torch.empty((6, HQ), device="cuda")
    positions = torch.cat([torch.arange(n - 3, n) for n in lens]).cuda()
    probs = torch.softmax(torch.randn((6, VOCAB), generator=s.g), -1).cuda()
    tokens, u, fu = torch.randint(0, VOCAB, (6,), generator=s.g).cuda(), torch.rand(6).cuda(), torch.rand(2).cuda()
    kept = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    got = torch.zeros(2, dtype=torch.int32, device="cuda")
    nxt = torch.zeros(2, dtype=torch.int64, device="cuda")
    m, cu = s.meta(rows, lens, counts)
    qlens = ints(counts, torch.int64)

    def enqueue():
        B.pa_rope_append_blocks(q=q, q_out=q_out, k=k, v=v, positions=positions, inv_freq=s.inv, cu_seqlens_q=cu,
                                cache_seqlens=m["cache_seqlens"], page_table=m["page_table"], max_seq_pages=MSP,
                                k_cache=s.k, v_cache=s.v, k_scale=s.ks, v_scale=s.vs)
        B.pa_decode_step_block(**m, seqlen_offset=0, max_seq_pages=MSP, q=q_out, k_cache=s.k, v_cache=s.v,
                               k_scale=s.ks, v_scale=s.vs, sm_scale=SCALE, out=out, lse=lse, cu_seqlens_q=cu,
                               max_q_len=3, qlens=qlens, q_mode=B.PA_Q_MODE_CUMSUM, workspace=s.ws)
        B.pa_verify_drafts(target_probs=probs, tokens=tokens, cu_seqlens_q=cu, cache_seqlens=m["cache_seqlens"],
                           uniforms=u, final_uniforms=fu, max_q_len=3, kept=kept, counts=got, next_tokens=nxt)

    results = lambda: [x.clone() for x in (out, lse, kept, got, nxt, s.k.view(torch.uint8), s.v.view(torch.uint8))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        enqueue()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            enqueue()
    for turn in range(3):
        d.copy_(s.inputs(6))
        tokens.copy_(torch.randint(0, VOCAB, (6,), generator=s.g))
        torch.cuda.synchronize()
        kv = [x.clone() for x in (s.k.view(torch.uint8), s.v.view(torch.uint8), s.ks, s.vs)]
        enqueue()
        torch.cuda.synchronize()
        want = results()
        for x, y in zip((s.k.view(torch.uint8), s.v.view(torch.uint8), s.ks, s.vs), kv):
            x.copy_(y)
        for x in (out, lse, kept, got, nxt):
            x.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, results()):
            assert torch.equal(x, y)
