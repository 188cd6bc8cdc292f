"""Pins of the cached-decoding oracle: library attention, closed forms, brute force."""
import itertools

import numpy as np
import pytest
import torch

from oracle import cached as OC


def _pools(rng, B, lengths, page, Hkv, d, extra=1):
    counts = [-(-n // page) for n in lengths]
    ids = rng.permutation(sum(counts) + extra)
    width = max(max(counts), 1)
    table = np.full((B, width), 0, dtype=np.int64)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = ids[at:at + c]
        at += c
    shape = (len(ids), page, Hkv, d)
    return rng.standard_normal(shape), rng.standard_normal(shape), table


def test_paged_attention_is_library_attention_on_the_gathered_slots():
    rng = np.random.default_rng(0)
    lengths, page, Hq, Hkv, d = [7, 1, 12], 5, 4, 2, 8
    k, v, table = _pools(rng, 3, lengths, page, Hkv, d)
    q = rng.standard_normal((3, Hq, d))
    kn, vn = rng.standard_normal((3, Hkv, d)), rng.standard_normal((3, Hkv, d))
    before = rng.random((3, 15))
    out, lse, mass = OC.paged_attention(q, k, v, table, lengths, kn, vn, before)
    for b, n in enumerate(lengths):
        rows = [(table[b, j // page], j % page) for j in range(n)]
        assert np.array_equal(k[rows[-1]], kn[b]) and np.array_equal(v[rows[-1]], vn[b])
        kk = torch.tensor(np.stack([k[r] for r in rows])).repeat_interleave(Hq // Hkv, 1)
        vv = torch.tensor(np.stack([v[r] for r in rows])).repeat_interleave(Hq // Hkv, 1)
        qq = torch.tensor(q[b])[:, None]
        want = torch.nn.functional.scaled_dot_product_attention(qq, kk.transpose(0, 1), vv.transpose(0, 1))
        assert np.allclose(out[b], want[:, 0].numpy(), atol=1e-12)
        # masses: one query head's worth of weight in all, on top of what was there
        kept = before[b, :n].copy()
        kept[-1] = 0.0
        assert np.isclose((mass[b, :n] - kept).sum(), 1.0)
        assert np.array_equal(mass[b, n:], before[b, n:])


def test_paged_attention_closed_forms():
    # equal keys: uniform weights; lse = s + log n
    k = np.ones((2, 4, 1, 8))
    v = np.arange(8.0)[:, None] * np.ones((8, 8))
    v = v.reshape(2, 4, 1, 8)
    out, lse, mass = OC.paged_attention(np.ones((1, 1, 8)), k, v, np.array([[1, 0]]), [6],
                                        mass=np.zeros((1, 8)), scale=0.5)
    assert np.allclose(out, np.mean([4, 5, 6, 7, 0, 1]))
    assert np.allclose(lse, 4.0 + np.log(6))
    assert np.allclose(mass, [[1 / 6] * 6 + [0, 0]])
    # a hole takes its slots out; only holes, or no slots, leave nothing
    out, lse, mass = OC.paged_attention(np.ones((1, 1, 8)), k, v, np.array([[1, -1]]), [6],
                                        mass=np.zeros((1, 8)))
    assert np.allclose(out, 5.5) and np.allclose(mass, [[0.25] * 4 + [0] * 4])
    for table, n in (([[-1, -1]], 6), ([[1, 0]], 0)):
        out, lse, _ = OC.paged_attention(np.ones((1, 1, 8)), k, v, np.array(table), [n])
        assert np.all(out == 0) and np.all(lse == -np.inf)


def test_evict_by_brute_force():
    rng = np.random.default_rng(1)
    for trial in range(200):
        n = int(rng.integers(1, 9))
        mass = rng.integers(0, 4, n).astype(float)  # many equal masses
        pos = rng.permutation(n)
        budget = int(rng.integers(1, 9))
        sink = int(rng.integers(0, budget + 1))
        recent = int(rng.integers(0, budget - sink + 1))
        src = OC.evict_one(mass, pos, budget, sink, recent)
        left = min(n, budget)
        assert len(src) == left and len(set(src)) == left
        safe = {j for j in range(n) if pos[j] < sink or pos[j] > n - 1 - recent}
        if n > budget:
            assert safe <= set(src)
            # no set of the same size that holds the protected slots weighs more
            best = max(sum(mass[list(c)]) for c in itertools.combinations(range(n), left)
                       if safe <= set(c))
            assert sum(mass[src]) == best
            # of equal masses the lower slot stays
            for a in set(src) - safe:
                for out in set(range(n)) - set(src):
                    assert mass[a] > mass[out] or a < out
        # slots that stay below the new length do not move, the others keep their order
        assert all(src[j] == j for j in range(left) if j in src)
        moved = [j for j in src if j >= left]
        assert moved == sorted(moved)


def test_evict_orders_nan_last_and_caps_protection():
    nan = float("nan")
    assert OC.evict_one([nan, -np.inf, 0.0], [0, 1, 2], 2, 0, 0) == [2, 1]
    assert OC.evict_one([0, 0, 0, 9.0], [0, 0, 0, 0], 2, 1, 1) == [0, 1]  # all protected


@pytest.mark.parametrize("K,V", [(1, 5), (3, 4), (4, 7)])
def test_beam_select_by_brute_force(K, V):
    rng = np.random.default_rng(K)
    for trial in range(50):
        x = rng.integers(-2, 3, (K, V)).astype(float)
        score = rng.integers(-2, 1, K).astype(float)
        done = (rng.random(K) < 0.3).astype(np.uint8)
        eos = int(rng.integers(-1, V))
        parent, token, out, ended = OC.beam_select(x, score, done, eos)
        logp = x - torch.logsumexp(torch.tensor(x), 1, keepdim=True).numpy()
        cands = {}
        for k in range(K):
            if done[k]:
                cands[(k, eos)] = score[k]
            else:
                for v in range(V):
                    cands[(k, v)] = score[k] + logp[k, v]
        best = sorted(cands.items(), key=lambda c: -c[1])[:K]
        assert np.allclose(out[:len(best)], [c[1] for c in best], atol=1e-12)
        assert len({(p, t) for p, t in zip(parent, token) if p >= 0}) == len(best)
        for p, t, s, e in zip(parent, token, out, ended):
            if p >= 0:
                assert np.isclose(cands[(p, t)], s) and e == (done[p] or t == eos)
            else:
                assert t == -1 and s == -np.inf and e == 0
        assert np.all(np.diff(out[:len(best)]) <= 0)


def test_beam_select_ties_banned_and_empty():
    parent, token, out, _ = OC.beam_select(np.zeros((2, 3)), np.zeros(2))
    assert parent.tolist() == [0, 0] and token.tolist() == [0, 1]
    x = np.array([[-np.inf, np.nan, 1.0], [0.0, 0.0, 0.0]])
    parent, token, out, _ = OC.beam_select(x, np.array([0.0, -np.inf]))
    assert parent.tolist() == [0, -1] and token.tolist() == [2, -1]
    assert out[0] == 0.0 and out[1] == -np.inf  # banned tokens leave the sum, too


def test_fork_keeps_every_beam_s_history():
    rng = np.random.default_rng(3)
    B, K, page, layers = 2, 3, 4, 2
    N = B * K
    lengths = np.array([4, 4, 4, 7, 7, 7])
    width, pages = 3, 40
    k = rng.standard_normal((layers, pages, page, 1, 2))
    v = rng.standard_normal((layers, pages, page, 1, 2))
    ids = rng.permutation(pages)
    table = ids[:N * width].reshape(N, width)
    fresh = ids[N * width:N * width + N]
    parent = np.array([[2, 2, -1], [0, 5, 1]])
    out = np.full((N, width), -7)
    want = []
    for p, n in zip(OC.parents(parent, K), range(N)):
        want.append([k[:, table[p, j // page], j % page].copy() for j in range(lengths[p])])
    got = OC.fork(parent, K, table, lengths, fresh, k, v, out)
    assert OC.parents(parent, K) == [2, 2, 2, 3, 4, 4]
    for n in range(N):
        rows = [k[:, out[n, j // page], j % page] for j in range(got[n])]
        assert np.array_equal(np.array(rows), np.array(want[n]))
        assert out[n, got[n] // page] == fresh[n]
        assert all(out[n, got[n] // page + 1:] == -7)
