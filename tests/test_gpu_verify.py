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
