"""The compositions' own bookkeeping (cached_decode.py) on the CPU: the library's calls are
played by the oracle's definitions, sequence by sequence."""
import numpy as np
import pytest
import torch

from oracle import cached as OC
from speculative_verification_cover_b200 import build, dd
from speculative_verification_cover_b200.cached_decode import BeamDecode, BudgetedCache


def _attention(q, cache, lengths, out, lse=None, k_new=None, v_new=None, **kw):
    """The append alone: these tests look at what the caches hold."""
    for n, m in enumerate(lengths.tolist()):
        assert 0 < m <= cache.slots
        page, row = int(cache.page_table[n, (m - 1) // cache.page_size]), (m - 1) % cache.page_size
        assert 0 <= page < cache.n_pages
        cache.k[page, row], cache.v[page, row] = k_new[n], v_new[n]


def _fork(cache, parent, lengths, fresh, table_out, lengths_out):
    out = table_out.numpy()
    lengths_out.copy_(torch.tensor(OC.fork(parent.numpy(), parent.shape[1], cache.page_table.numpy(), lengths.numpy(),
                                           fresh.numpy(), cache.k.numpy(), cache.v.numpy(), out)))


def _reorder(parent, states):
    rows = OC.parents(parent.numpy(), parent.shape[1])
    for src, dst in states:
        dst.view(len(rows), -1).copy_(src.view(len(rows), -1)[rows])


@pytest.fixture
def played(monkeypatch):
    build.build()
    rng = np.random.default_rng(5)

    def select(logits, score, parent, token, score_out, done=None, done_out=None, **kw):
        parent.copy_(torch.tensor(rng.integers(0, parent.shape[1], parent.shape)))
        token.copy_(torch.tensor(rng.integers(0, 50, token.shape)))
        score_out.copy_(score)
        done_out.copy_(done)

    for name, f in (("_gpu", lambda t, name: -1), ("dd_paged_attention", _attention), ("dd_paged_fork", _fork),
                    ("dd_beam_reorder", _reorder), ("dd_beam_select", select)):
        monkeypatch.setattr(dd, name, f)


PATTERNS = {"begin first": lambda i: "ba", "advance first": lambda i: "ab", "several tokens a choice": lambda i: "bba",
            "several choices a token": lambda i: "baa", "mixed": lambda i: ("ab", "bbba", "aab", "a", "b")[i % 5]}


def beams_hold_their_histories(pattern, page, L, device):
    """Every beam's slots, followed through its table, are its own history."""
    layers, B, K, Hkv, d, V, steps = 2, 2, 3, 1, 64, 52, 13
    gen = torch.Generator().manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    k, v = rnd(layers, B, L, Hkv, d), rnd(layers, B, L, Hkv, d)
    dec = BeamDecode(k.to(device), v.to(device), 1, K, V, steps, page_size=page)
    N = B * K
    hist = [torch.stack([k[:, n // K], v[:, n // K]], 2) for n in range(N)]  # [layers, slots, 2, Hkv, d]
    toks = torch.zeros(N, 0, dtype=torch.int32)
    begun = chosen = 0
    for op in "".join(PATTERNS[pattern](i) for i in range(20)):
        if op == "b" and begun < steps:
            dec.begin()
            begun += 1
            new = rnd(2, layers, N, Hkv, d)
            for l in range(layers):
                dec.attend(l, torch.zeros(N, 1, d, device=device), new[0, l].to(device), new[1, l].to(device))
            hist = [torch.cat([h, new[:, :, n].transpose(0, 1)[:, None]], 1) for n, h in enumerate(hist)]
        elif op == "a" and chosen < steps:
            dec.advance(rnd(B, K, V).to(device))
            chosen += 1
            rows = OC.parents(dec.parent.cpu().numpy(), K)
            hist = [hist[p] for p in rows]
            toks = torch.cat([toks[rows], dec.token.view(N, 1).cpu()], 1)
            assert torch.equal(dec.tokens.view(N, -1)[:, :chosen].cpu(), toks)
        table, j = dec.table.cpu().long(), torch.arange(L + begun)
        pools = [p.cpu() for p in (dec.pool_k, dec.pool_v)]
        assert dec.lengths.tolist() == [L + begun] * N
        for n in range(N):
            held = torch.stack([p[:, table[n, j // page], j % page] for p in pools], 2)
            assert torch.equal(held, hist[n]), (begun, chosen, n)
    assert begun == steps or chosen == steps
    for call, all_taken in ((dec.begin, begun == steps), (lambda: dec.advance(rnd(B, K, V).to(device)), chosen == steps)):
        if all_taken:
            with pytest.raises(ValueError, match="steps"):
                call()


@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("page,L", [(1, 3), (2, 4), (2, 5), (3, 9), (4, 10), (16, 5)])
def test_beams_hold_their_own_histories(played, pattern, page, L):
    """Whatever the order of new tokens (begin, attend) and choices (advance): a prompt's logits
    may be chosen from before the first token, and tokens may follow each other unbranched."""
    beams_hold_their_histories(pattern, page, L, "cpu")


def test_budgets_and_lengths_out_of_range(played, monkeypatch):
    """What would send a slot's position behind its row is refused, or clamped as the library
    clamps lengths."""
    make = lambda **kw: BudgetedCache(**(dict(N=3, Hq=2, Hkv=1, d=64, budget=16, page_size=4, sink=2, recent=6,
                                              device="cpu", dtype=torch.float32) | kw))
    for kw in (dict(every=0), dict(every=-1), dict(budget=0), dict(budget=7), dict(sink=-1), dict(recent=-1),
               dict(sink=4, recent=13), dict(prompt=-1)):
        with pytest.raises(ValueError):
            make(**kw)
    make(budget=8), make(sink=16, recent=0)
    evicted = []

    def evict(cache, lengths, mass, pos, budget, mass_out, pos_out, lengths_out, **kw):
        evicted.append(lengths.tolist())
        mass_out.copy_(mass), pos_out.copy_(pos), lengths_out.copy_(lengths.clamp(max=budget))

    monkeypatch.setattr(dd, "dd_cache_evict", evict)
    c = make(every=2)
    k, q, new = torch.randn(3, 10, 1, 64), torch.zeros(3, 2, 64), torch.randn(3, 1, 64)
    c.fill(k, k, lengths=torch.tensor([-4, 1000, 7], dtype=torch.int32))
    assert c.lengths.tolist() == c.seen.tolist() == [0, 10, 7]
    for t in range(12):
        c.attend(q, new, new)
        n = c.lengths.tolist()
        assert max(n) <= c.cache.slots and c.pos[1, n[1] - 1] == 10 + t and c.pos[0, n[0] - 1] == t
    assert evicted == [[8, 18, 15], [10, 18, 17]]
