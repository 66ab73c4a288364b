"""GPU parity of the draft verification against the definition in verify_reference.py: accepted
rows and tokens equal, for chains and trees, with and without draft probabilities."""

import random

import pytest
import torch

import verify_reference as R
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


class Drafts:
    """Probabilities, tokens and trees of a batch; `width` siblings at most (0: chains)."""

    def __init__(self, q_lens, vocab, width, drafted, seed, spread=2.0, pad=0):
        g = torch.Generator().manual_seed(seed)
        r = random.Random(seed)
        self.q_lens, self.vocab, self.drafted = q_lens, vocab, drafted
        rows = sum(q_lens)
        x = torch.randn((rows, vocab), generator=g) * spread
        self.target = torch.softmax(x, -1)
        self.draft = torch.softmax(x + torch.randn((rows, vocab), generator=g), -1) if drafted else None
        self.parents, tokens = [], []
        at = 0
        for d in q_lens:
            for i in range(d):
                up = i - 1 if width == 0 else r.randint(max(0, i - width), i - 1) if i else -1
                self.parents.append(up)
                if i == 0:
                    tokens.append(-5)  # (not looked at)
                    continue
                like = self.draft if drafted else self.target
                top = torch.multinomial(like[at + up], 1, generator=g) if drafted else \
                    torch.topk(like[at + up], min(4, vocab)).indices[torch.randint(min(4, vocab), (1,), generator=g)]
                tokens.append(int(top))
            at += d
        self.chain = width == 0
        self.tokens = torch.tensor(tokens, dtype=torch.int64)
        self.uniforms = torch.rand((rows,), generator=g)
        self.final = torch.rand((len(q_lens),), generator=g)
        self.n = torch.tensor([d + r.randint(0, 500) for d in q_lens], dtype=torch.int32)
        self.pad = pad

    def on_device(self, x):
        """Rows on the device, `pad` columns apart."""
        wide = torch.full((x.shape[0], self.vocab + self.pad), 9.0, device="cuda")
        wide[:, :self.vocab] = x
        return wide[:, :self.vocab]

    def run(self, **over):
        bs, mql = len(self.q_lens), max(max(self.q_lens), 1)
        cu = torch.zeros(bs + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(self.q_lens), 0)
        full = lambda *s, dt=torch.int32: torch.full(s, 77, dtype=dt, device="cuda")
        kw = dict(target_probs=self.on_device(self.target),
                  draft_probs=self.on_device(self.draft) if self.drafted else None,
                  tokens=self.tokens.cuda(),
                  parents=None if self.chain else torch.tensor(self.parents, dtype=torch.int32).cuda(),
                  cu_seqlens_q=cu.cuda(), cache_seqlens=self.n.cuda(), uniforms=self.uniforms.cuda(),
                  final_uniforms=self.final.cuda(), max_q_len=mql, kept=full(bs, mql + 2),
                  counts=full(bs), begin=full(bs), next_tokens=full(bs, dt=torch.int64)) | over
        B.pa_verify_drafts(**kw)
        torch.cuda.synchronize()
        return tuple(None if kw[x] is None else kw[x].cpu() for x in ("kept", "counts", "begin", "next_tokens"))

    def check(self, got):
        kept, counts, begin, tokens = got
        at = 0
        accepted = 0
        for b, d in enumerate(self.q_lens):
            base = int(self.n[b]) - d
            if d:
                rows = slice(at, at + d)
                path, token = R.verify(self.target[rows].numpy(), self.draft[rows].numpy() if self.drafted else None,
                                       self.tokens[rows].tolist(), self.parents[rows],
                                       self.uniforms[rows].tolist(), float(self.final[b]))
            else:
                path, token = [], -1
            accepted += len(path)
            want = [base + i for i in path]
            assert kept[b].tolist() == want + [-1] * (kept.shape[1] - 2 - len(want)) + [77, 77]
            assert int(counts[b]) == len(path) and int(begin[b]) == base
            assert int(tokens[b]) == (-1 if token is None else token)
            at += d
        return accepted


CASES = [  # q_lens, vocab, width (0: chain), drafted, row padding
    ([5], 32000, 0, True, 0),
    ([1], 1, 0, True, 0),
    ([1, 1, 1], 50, 0, False, 3),
    ([4, 0, 9, 1], 1000, 0, True, 0),
    ([9] * 12, 4096, 0, True, 0),
    ([7, 3], 100003, 0, False, 0),
    ([12, 30, 1], 517, 3, True, 5),
    ([16] * 10, 300, 6, True, 0),
    ([40, 256], 2000, 8, True, 0),
    ([33, 64, 2], 10007, 5, False, 0),
    ([200], 8, 9, False, 0),
    ([64] * 8, 3, 5, True, 1),
    ([10] * 6, 131072, 4, False, 0),
]


@pytest.mark.parametrize("q_lens,vocab,width,drafted,pad", CASES)
def test_verify(q_lens, vocab, width, drafted, pad):
    d = Drafts(q_lens, vocab, width, drafted, seed=vocab + width, pad=pad)
    got = d.run()
    d.check(got)
    again = d.run()
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_accepted_tokens_follow_the_target():
    """20000 requests of one drafted token over 12 tokens: whatever the draft, the first token that
    comes out is the target's to 5 standard deviations of its count."""
    n, vocab = 20000, 12
    g = torch.Generator().manual_seed(5)
    p = torch.softmax(torch.randn(vocab, generator=g) * 1.5, -1)
    q = torch.softmax(torch.randn(vocab, generator=g) * 1.5, -1)
    for drafted in (True, False):
        d = Drafts([2] * n, vocab, 0, drafted, seed=6)
        d.target = p.expand(2 * n, vocab).contiguous()
        d.draft = q.expand(2 * n, vocab).contiguous() if drafted else None
        x = torch.multinomial(q, n, replacement=True, generator=g)
        d.tokens = torch.stack((torch.zeros(n, dtype=torch.int64), x), 1).flatten()
        kept, counts, begin, tokens = d.run()
        first = torch.where(counts == 2, x, tokens)
        seen = torch.bincount(first, minlength=vocab).double()
        want = p.double() * n
        assert ((seen - want).abs() <= 5 * (want * (1 - p.double())).sqrt() + 1).all()


def test_trees_with_siblings_follow_the_target():
    """Three siblings drawn from the draft, and the three likeliest tokens: the token that follows
    the root is the target's."""
    n, vocab = 20000, 9
    g = torch.Generator().manual_seed(7)
    p = torch.softmax(torch.randn(vocab, generator=g), -1)
    q = torch.softmax(torch.randn(vocab, generator=g), -1)
    for drafted in (True, False):
        d = Drafts([4] * n, vocab, 3, drafted, seed=8)
        d.parents = [-1, 0, 0, 0] * n
        d.target = p.expand(4 * n, vocab).contiguous()
        d.draft = q.expand(4 * n, vocab).contiguous() if drafted else None
        x = torch.multinomial(q, 3 * n, replacement=True, generator=g).view(n, 3) if drafted else \
            torch.topk(q, 3).indices.expand(n, 3)
        d.tokens = torch.cat((torch.zeros(n, 1, dtype=torch.int64), x), 1).flatten().contiguous()
        kept, counts, begin, tokens = d.run()
        node = (kept[:, 1] - begin).clamp(min=0).long()
        first = torch.where(counts == 2, d.tokens.view(n, 4).gather(1, node[:, None])[:, 0], tokens)
        seen = torch.bincount(first, minlength=vocab).double()
        want = p.double() * n
        assert ((seen - want).abs() <= 5 * (want * (1 - p.double())).sqrt() + 1).all()


def test_nothing_left_of_the_row():
    """A draft equal to the target is accepted for any number below 1; where a number of 1 rejects it
    all the same, the token comes from the row itself.  A row of zeros gives -1 and is reported."""
    d = Drafts([3, 2], 40, 0, True, seed=9)
    d.draft = d.target.clone()
    d.check(d.run())
    d.uniforms.fill_(1.0)
    d.check(d.run())
    d.target[3].zero_()
    d.target[4].zero_()
    d.check(d.run())
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_NO_PROBABILITY


def test_what_is_refused_is_reported():
    d = Drafts([4, 3, 5], 50, 3, False, seed=10)
    d.tokens[2], d.tokens[5] = 50, -1                        # outside the vocabulary: never accepted
    d.check(d.run())
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_TOKEN_OUT_OF_RANGE
    d = Drafts([4, 3, 5], 50, 3, True, seed=11)
    got = d.run(parents=torch.tensor([-1, 1, 0, 9, -1, 0, -2, -1, 0, 1, 2, 3], dtype=torch.int32).cuda())
    assert B.pa_read_error_flags(reset=True) == B.DEVERR_TREE_PARENT
    d.parents = [-1, -1, 0, -1, -1, 0, -1, -1, 0, 1, 2, 3]
    d.check(got)
    d.n[1] = 2                                               # fewer than its rows
    kept, counts, begin, tokens = d.run(max_q_len=4, kept=torch.full((3, 6), 77, dtype=torch.int32, device="cuda"))
    assert B.pa_read_error_flags(reset=True) & B.DEVERR_SEQLEN_OUT_OF_RANGE
    assert counts[1:].tolist() == [0, 0] and tokens[1:].tolist() == [-1, -1]
    assert kept[1:].tolist() == [[-1] * 4 + [77, 77]] * 2 and int(counts[0]) > 0


def test_without_lengths_kept_are_rows():
    d = Drafts([6, 6], 100, 0, True, seed=12)
    with_lengths = d.run()
    d.n = torch.tensor([6, 6], dtype=torch.int32)
    kept, counts, begin, tokens = d.run(cache_seqlens=None, begin=None)
    assert begin is None and torch.equal(counts, with_lengths[1]) and torch.equal(tokens, with_lengths[3])
    for b in range(2):
        assert kept[b, :int(counts[b])].tolist() == list(range(int(counts[b])))


def test_verified_path_compacts_the_cache():
    """kept, counts and begin go to pa_compact_cache as they are."""
    d = Drafts([12, 9], 30, 4, False, seed=13)
    kept, counts, begin, tokens = d.run()
    d.check((kept, counts, begin, tokens))
    page, hkv = 16, 2
    per = [-(-int(n) // page) for n in d.n]
    table = torch.zeros((2, max(per)), dtype=torch.int32)
    table[0, :per[0]] = torch.arange(per[0])
    table[1, :per[1]] = torch.arange(per[0], sum(per))
    k, v = (torch.randn((sum(per), hkv, page, 128)).to(torch.bfloat16).cuda() for _ in "kv")
    before = k.clone()
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    B.pa_compact_cache(page_table=table.cuda(), cache_seqlens=d.n.cuda(), kept=kept[:, None, :12].contiguous().cuda(),
                       counts=counts.cuda(), begin=begin.cuda(), k_cache=k, v_cache=v, max_seq_pages=max(per),
                       new_seqlens=new)
    torch.cuda.synchronize()
    assert torch.equal(new.cpu(), begin + counts)
    for b in range(2):
        for i in range(int(counts[b])):
            src, dst = int(kept[b, i]), int(begin[b]) + i
            assert torch.equal(k[table[b, dst // page].item(), :, dst % page],
                               before[table[b, src // page].item(), :, src % page])


@pytest.mark.parametrize("vocab,new", [(1, 1), (7, 2), (40, 3)])
def test_blocks_that_start_late(vocab, new):
    """More clusters than the GPU holds at once, with rows so short that a block has its sum as soon
    as it starts, every fifth request without rows: the sums of blocks that start later are there."""
    n = 3000
    d = Drafts([0 if b % 5 == 4 else new for b in range(n)], vocab, 0, True, seed=21)
    first = d.run()
    d.check(first)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(first, d.run()))


@pytest.mark.parametrize("drafted", [True, False])
def test_a_batch_without_rows(drafted):
    """Every request of a padded batch without rows: the tensors of rows are empty."""
    d = Drafts([0, 0, 0], 50, 0, drafted, seed=22)
    d.check(d.run())
    kept, counts, begin, tokens = d.run(max_q_len=4, kept=torch.full((3, 6), 77, dtype=torch.int32, device="cuda"))
    assert kept.tolist() == [[-1] * 4 + [77, 77]] * 3
    assert counts.tolist() == [0] * 3 and tokens.tolist() == [-1] * 3 and torch.equal(begin, d.n)
