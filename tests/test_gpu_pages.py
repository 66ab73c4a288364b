"""The page operators on the GPU against a plain model of their state: tables, holders and
every byte of the pools equal after each call."""

import random

import pytest
import torch

from paged_kv_decode_metadata_gb300 import binding as B
from paged_kv_decode_metadata_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    B.load()
    B.pa_read_error_flags(reset=True)
    yield
    assert B.pa_read_error_flags(reset=True) == 0


def pool(shape, dtype, g):
    x = torch.randint(0, 120, shape, generator=g, dtype=torch.uint8)
    return x.to(dtype) if dtype != torch.float8_e4m3fn else x.view(dtype)


class Pages:
    """The state twice: a plain one on the CPU and the library's."""

    def __init__(self, rows, num_pages, page, msp, pools, seed=0, stride=None):
        g = torch.Generator().manual_seed(seed)
        self.page, self.msp, self.num_pages = page, msp, num_pages
        width = stride or msp * page
        self.table = torch.full((rows, width), -7, dtype=torch.int32)
        self.refs = torch.zeros(num_pages, dtype=torch.int32)
        self.pools = [pool((num_pages, *shape), dtype, g) for shape, dtype in pools]
        self.lens = [0] * rows
        self.d_table, self.d_refs = self.table.cuda(), self.refs.cuda()
        self.d_pools = [x.cuda() for x in self.pools]

    def common(self, rows, lens):
        return dict(req_to_token=self.d_table, page_refs=self.d_refs, page_size=self.page,
                    max_seq_pages=self.msp, lens=torch.tensor(lens, dtype=torch.int32).cuda()), \
            torch.tensor(rows, dtype=torch.int64).cuda()

    def workspace(self, count):
        return torch.full((B.pa_pages_workspace_bytes(self.num_pages, count),), 0xff, dtype=torch.uint8,
                          device="cuda")

    def free_pages(self):
        return [i for i in range(self.num_pages) if self.refs[i] == 0]

    def hand_out(self, row, at, page):
        lo = at * self.page
        hi = min(lo + self.page, self.table.shape[1])
        self.table[row, lo:hi] = torch.arange(page * self.page, page * self.page + hi - lo, dtype=torch.int32)

    def page_at(self, row, at):
        return int(self.table[row, at * self.page]) // self.page

    def check(self):
        torch.cuda.synchronize()
        assert torch.equal(self.d_table.cpu(), self.table)
        assert torch.equal(self.d_refs.cpu(), self.refs)
        for a, b in zip(self.d_pools, self.pools):
            assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))

    def extend(self, rows, new_lens):
        old = [self.lens[r] for r in rows]
        free, at, want = self.free_pages(), 0, []
        for r, a, b in zip(rows, old, new_lens):
            first, need = -(-a // self.page), max(0, -(-b // self.page) - -(-a // self.page))
            got = min(need, len(free) - at)
            for k in range(got):
                self.hand_out(r, first + k, free[at + k])
                self.refs[free[at + k]] = 1
            at += got
            want.append(max(a, b) if got == need else (first + got) * self.page)
            self.lens[r] = want[-1]
        kw, d_rows = self.common(rows, old)
        granted = torch.full((len(rows),), -9, dtype=torch.int32, device="cuda")
        B.pa_pages_extend(rows=d_rows, new_lens=torch.tensor(new_lens, dtype=torch.int32).cuda(),
                          granted=granted, workspace=self.workspace(len(rows)), **kw)
        self.check()
        assert granted.tolist() == want
        return want

    def fork(self, parents, children, lens):
        free, at, want = self.free_pages(), 0, []
        for s, c, n in zip(parents, children, lens):
            full = n // self.page
            got = n
            for k in range(full):
                self.hand_out(c, k, self.page_at(s, k))
                self.refs[self.page_at(s, k)] += 1
            if n % self.page:
                if at < len(free):
                    new, src = free[at], self.page_at(s, full)
                    at += 1
                    self.refs[new] = 1
                    self.hand_out(c, full, new)
                    for x in self.pools:
                        x.view(torch.uint8)[new] = x.view(torch.uint8)[src]
                else:
                    got = full * self.page
            want.append(got)
            self.lens[c] = got
        kw, d_parents = self.common(parents, lens)
        child_lens = torch.full((len(parents),), -9, dtype=torch.int32, device="cuda")
        B.pa_pages_fork(parents=d_parents, children=torch.tensor(children).cuda(), pools=self.d_pools,
                        child_lens=child_lens, workspace=self.workspace(len(parents)), **kw)
        self.check()
        assert child_lens.tolist() == want

    def free(self, rows, keep=None):
        lens = [self.lens[r] for r in rows]
        for i, r in enumerate(rows):
            k = keep[i] if keep else 0
            for at in range(-(-k // self.page), -(-lens[i] // self.page)):
                if self.table[r, at * self.page] >= 0:
                    self.refs[self.page_at(r, at)] -= 1
                    self.table[r, at * self.page] = -1
            self.lens[r] = min(k, lens[i])
        kw, d_rows = self.common(rows, lens)
        B.pa_pages_free(rows=d_rows, keep_lens=torch.tensor(keep, dtype=torch.int32).cuda() if keep else None, **kw)
        self.check()

    def compact(self, rows):
        live = [i for i in range(self.num_pages) if self.refs[i] > 0]
        moves = dict(zip([i for i in live if i >= len(live)],
                         [i for i in range(len(live)) if self.refs[i] == 0]))
        for src, dst in moves.items():
            for x in self.pools:
                x.view(torch.uint8)[dst] = x.view(torch.uint8)[src]
            self.refs[dst], self.refs[src] = self.refs[src].item(), 0
        for r in set(rows):
            for at in range(-(-self.lens[r] // self.page)):
                if self.table[r, at * self.page] >= 0 and self.page_at(r, at) in moves:
                    self.hand_out(r, at, moves[self.page_at(r, at)])
        kw, d_rows = self.common(rows, [self.lens[r] for r in rows])
        page_map = torch.full((self.num_pages,), -9, dtype=torch.int32, device="cuda")
        num_live = torch.full((1,), -9, dtype=torch.int32, device="cuda")
        B.pa_pages_compact(rows=d_rows, pools=self.d_pools, page_map=page_map, num_live=num_live,
                           workspace=self.workspace(len(rows)), **kw)
        self.check()
        assert int(num_live) == len(live)
        want = [-1] * self.num_pages
        for i in live:
            want[i] = moves.get(i, i)
        assert page_map.tolist() == want


BF16 = [((2, 16, 128), torch.bfloat16)] * 2
FP8 = [((3, 16, 128), torch.float8_e4m3fn), ((3, 1), torch.float32)] * 2


@pytest.mark.parametrize("num_pages,page,msp,pools,stride", [
    (40, 16, 9, BF16, None),
    (300, 16, 20, FP8, 20 * 16 + 5),
    (64, 7, 12, [((1,), torch.float32), ((5, 3), torch.int32), ((4000,), torch.float32)], 12 * 7 - 3),
    (5000, 64, 30, [((34,), torch.int16)], None),
    (50, 1, 40, [((2, 128), torch.bfloat16)] * 131, None),   # more pools than one launch takes
])
def test_sequences(num_pages, page, msp, pools, stride):
    """Requests that grow, fork, shrink, end, and are packed, in seeded sequences."""
    rng = random.Random(num_pages)
    rows = 12
    s = Pages(rows, num_pages, page, msp, pools, seed=page, stride=stride)
    cap = min(msp * page, s.table.shape[1])
    for _ in range(14):
        idle = [r for r in range(rows) if s.lens[r] == 0]
        busy = [r for r in range(rows) if s.lens[r] > 0]
        what = rng.choice(["extend", "extend", "fork", "free", "trim", "compact"])
        if what == "extend":
            pick = rng.sample(range(rows), 4)
            room = len(s.free_pages()) * page // 6
            s.extend(pick, [min(cap, s.lens[r] + rng.randint(0, max(1, room))) for r in pick])
        elif what == "fork" and busy and idle and len(s.free_pages()) >= len(idle):
            parents = [rng.choice(busy) for _ in idle]
            s.fork(parents, rng.sample(idle, len(idle)), [rng.randint(0, s.lens[p]) for p in parents])
        elif what == "free" and busy:
            pick = rng.sample(busy, rng.randint(1, len(busy)))
            s.free(pick + pick[:1])            # a row listed twice is given back once
        elif what == "trim" and busy:
            s.free(busy, [rng.randint(0, s.lens[r]) for r in busy])
        elif what == "compact":
            s.compact(busy + busy[:1] if busy else [0])
    s.free(list(range(rows)))
    assert int(s.refs.sum()) == 0


def test_many_requests():
    """More entries than one round of the plan's scan; shared prefixes of 1500 children."""
    s = Pages(1601, 3000, 16, 4, [((8,), torch.float32)])
    s.extend([0], [41])
    s.fork([0] * 1500, list(range(1, 1501)), [41 - i % 3 * 9 for i in range(1500)])
    s.extend(list(range(1501, 1600)), [50 + i % 15 for i in range(99)])
    s.free(list(range(0, 1500, 2)))
    s.compact(list(range(1601)))


def test_out_of_pages_serves_in_order():
    s = Pages(6, 7, 16, 6, BF16)
    assert s.extend([0, 1, 2, 3], [40, 33, 20, 5]) == [40, 33, 16, 0]
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_OUT_OF_PAGES
    s.fork([0, 1], [4, 5], [40, 32])       # no page for the partly filled one: its full pages
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_OUT_OF_PAGES
    assert s.lens[4] == 32 and s.lens[5] == 32


def test_pages_between_pools_and_pinned_memory():
    g = torch.Generator().manual_seed(3)
    a = [pool((9, 4, 16, 128), torch.bfloat16, g).cuda(), pool((9, 4), torch.float32, g).cuda()]
    host = [torch.zeros((5, 4, 16, 128), dtype=torch.bfloat16).pin_memory(), torch.zeros((5, 4)).pin_memory()]
    idx = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()
    B.pa_pages_copy(src_pools=a, dst_pools=host, src_pages=idx(8, 0, -1, 3), dst_pages=idx(0, 4, 2, 1))
    torch.cuda.synchronize()
    for x, y in zip(a, host):
        assert torch.equal(y[[0, 4, 1]], x.cpu()[[8, 0, 3]]) and not y[[2, 3]].any()
    B.pa_pages_copy(src_pools=host, dst_pools=a, src_pages=idx(0, 1), dst_pages=idx(5, 6))
    before = [x.clone() for x in a]
    B.pa_pages_copy(src_pools=a, src_pages=idx(5, 7, 2), dst_pages=idx(1, -1, 4))
    torch.cuda.synchronize()
    for x, w in zip(a, before):
        w[[1, 4]] = w[[5, 2]]
        assert torch.equal(x, w) and torch.equal(x[5].cpu(), x[8].cpu())


def test_what_the_device_alone_sees_is_refused_and_reported():
    s = Pages(4, 8, 16, 3, BF16)
    s.extend([0, 1], [40, 20])
    kw, _ = s.common([0], [40])
    rows = lambda *x: torch.tensor(x).cuda()
    ints = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()
    out = torch.full((2,), -9, dtype=torch.int32, device="cuda")
    B.pa_pages_fork(parents=rows(0, 9), children=rows(-1, 2), pools=s.d_pools, child_lens=out,
                    workspace=s.workspace(2), **kw | dict(lens=ints(40, 16)))
    assert out.tolist() == [0, 0] and B.pa_read_error_flags(reset=True) == B.DEVERR_POOL_ROW_OUT_OF_RANGE
    B.pa_pages_fork(parents=rows(0, 1), children=rows(2, 3), pools=s.d_pools, child_lens=out,
                    workspace=s.workspace(2), **kw | dict(lens=ints(49, -1)))
    assert out.tolist() == [0, 0] and B.pa_read_error_flags(reset=True) == B.DEVERR_SEQLEN_OUT_OF_RANGE
    B.pa_pages_extend(rows=rows(7, 1), new_lens=ints(10, 60), granted=out, workspace=s.workspace(2),
                      **kw | dict(lens=ints(0, 20)))
    assert out.tolist() == [0, 20]
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_POOL_ROW_OUT_OF_RANGE | B.DEVERR_SEQLEN_OUT_OF_RANGE
    B.pa_pages_free(rows=rows(4, 0), **kw | dict(lens=ints(16, 1000)))
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_POOL_ROW_OUT_OF_RANGE | B.DEVERR_SEQLEN_OUT_OF_RANGE
    s.check()
    # a page that nobody holds, and one outside the pool
    s.d_table[3, 0] = s.table[3, 0] = 7 * 16
    s.d_table[3, 16] = s.table[3, 16] = 100 * 16
    B.pa_pages_free(rows=rows(3), **kw | dict(lens=ints(32)))
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_PAGE_REFS | B.DEVERR_PAGE_OUT_OF_RANGE
    s.table[3, 0] = s.table[3, 16] = -1
    s.check()


def test_columns_beside_a_table_stay():
    """A table that is a range of columns of a wider one, and one row of it: what lies beside stays."""
    big = torch.full((5, 100), 77, dtype=torch.int32, device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()
    rows = lambda *x: torch.tensor(x).cuda()
    refs = torch.zeros(12, dtype=torch.int32, device="cuda")
    pages = [torch.arange(12 * 8, dtype=torch.float32, device="cuda").view(12, 8)]
    out, one = ints(0, 0), ints(0)
    ws = torch.empty(B.pa_pages_workspace_bytes(12, 2), dtype=torch.uint8, device="cuda")
    kw = dict(req_to_token=big[:, 20:68], page_refs=refs, page_size=16, max_seq_pages=3)
    B.pa_pages_extend(rows=rows(0, 4), lens=ints(0, 0), new_lens=ints(40, 48), granted=out, workspace=ws, **kw)
    B.pa_pages_fork(parents=rows(0, 4), children=rows(1, 3), lens=ints(40, 48), pools=pages, child_lens=out,
                    workspace=ws, **kw)
    # one row, whose last page ends past its columns
    B.pa_pages_extend(rows=rows(0), lens=ints(0), new_lens=ints(30), granted=one, workspace=ws,
                      **kw | dict(req_to_token=big[2:3, 70:100], max_seq_pages=2))
    live = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    B.pa_pages_free(rows=rows(0, 4), lens=ints(40, 48), **kw)
    B.pa_pages_compact(rows=rows(1, 3), lens=ints(40, 48), pools=pages, page_map=torch.empty_like(refs),
                       num_live=live, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert out.tolist() == [40, 48] and one.tolist() == [30] and int(live) == 8
    mine = torch.zeros((5, 100), dtype=torch.bool)
    mine[[0, 1, 3, 4], 20:68] = True
    mine[2, 70:100] = True
    assert bool((big.cpu()[~mine] == 77).all())
    assert big[2, 70:100].tolist() == list(range(7 * 16, 8 * 16)) + list(range(8 * 16, 8 * 16 + 14))
    with pytest.raises(ValueError, match="room for fewer"):
        B.pa_pages_free(rows=rows(0), lens=ints(0), **kw | dict(req_to_token=big[:, 20:70], max_seq_pages=4))


@pytest.mark.parametrize("children", [2, 3, 500])
def test_pages_that_nobody_holds_are_not_forked(children):
    """Many children of a row with a full page, and a last one, that nobody holds: refused for all of
    them alike, whatever their order."""
    for last in (48, 40):                       # whole pages; a partly filled last one
        s = Pages(children + 2, children + 8, 16, 3, BF16)
        s.extend([0, 1], [last, 48])
        dead = [s.page_at(0, 1)] + ([s.page_at(0, 2)] if last == 40 else [])
        s.d_refs[dead] = 0
        kw, d_parents = s.common([0] * children, [last] * children)
        lens = torch.full((children,), -9, dtype=torch.int32, device="cuda")
        B.pa_pages_fork(parents=d_parents, children=torch.arange(2, children + 2).cuda(), pools=s.d_pools,
                        child_lens=lens, workspace=s.workspace(children), **kw)
        torch.cuda.synchronize()
        assert B.pa_read_error_flags(reset=True) == B.DEVERR_PAGE_REFS
        assert lens.tolist() == [48 if last == 48 else 32] * children
        s.refs[dead] = 0
        s.refs[s.page_at(0, 0)] += children
        s.table[2:, :16] = s.table[0, :16]
        s.table[2:, 16:32] = -1
        if last == 48:
            s.refs[s.page_at(0, 2)] += children
            s.table[2:, 32:] = s.table[0, 32:]
        s.check()


def test_a_row_cut_short_inside_a_shared_page():
    """Cut by a fork at its new length, a row has a page of its own to append to; cut by a free alone it
    goes on sharing the page, as the header says."""
    s = Pages(4, 12, 16, 4, BF16)
    s.extend([0], [60])
    s.fork([0], [1], [48])                      # three full pages shared
    s.fork([1], [2], [40])                      # row 1 cut to 40: its last page copied
    s.free([1])
    s.extend([2], [55])
    assert s.page_at(2, 2) != s.page_at(0, 2) and int(s.refs[s.page_at(2, 2)]) == 1
    assert int(s.refs[s.page_at(0, 2)]) == 1
    s.fork([0], [3], [48])
    s.free([3], [40])
    assert s.page_at(3, 2) == s.page_at(0, 2) and int(s.refs[s.page_at(0, 2)]) == 2
    s.free([0, 2, 3])
    assert int(s.refs.sum()) == 0
