"""The cached operators run together, as speculative_verification_cover_b200/cached_decode.py
composes them: every step against fp64 bookkeeping that never shares, moves or drops
anything it was not told to."""
import numpy as np
import pytest
import torch

from oracle import cached as OC
from speculative_verification_cover_b200 import dd
from speculative_verification_cover_b200.cached_decode import BeamDecode, BudgetedCache
from tests import cached_cases as CC
from tests.test_cached_compose import PATTERNS, beams_hold_their_histories

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,every,prompt", [(torch.bfloat16, 1, 40), (torch.float32, 5, 100), (torch.bfloat16, 3, 20)])
def test_budgeted_cache(dtype, every, prompt):
    N, Hq, Hkv, d, budget, steps = 3, 8, 2, 64, 48, 40
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(dtype)
    c = BudgetedCache(N, Hq, Hkv, d, budget, page_size=5, sink=2, recent=6, every=every, prompt=prompt,
                      dtype=dtype)
    k, v, mass = rnd(N, prompt, Hkv, d), rnd(N, prompt, Hkv, d), torch.rand(N, prompt, generator=gen)
    lengths = torch.tensor([prompt, prompt // 2, 1], dtype=torch.int32)
    c.fill(k.cuda(), v.cuda(), mass.cuda(), lengths.cuda())
    # the oracle's caches: per sequence a list of (position, k, v), by slot; the masses
    # follow the library's own between steps (fp32), so that a choice between two nearly
    # equal masses is the same on both sides
    held = [[(j, CC.bits64(k[n, j]), CC.bits64(v[n, j])) for j in range(int(lengths[n]))] for n in range(N)]
    masses = [mass[n, :int(lengths[n])].numpy() for n in range(N)]
    seen = lengths.tolist()

    def evict():
        for n in range(N):
            src = OC.evict_one(masses[n], np.array([h[0] for h in held[n]]), budget, 2, 6)
            held[n] = [held[n][j] for j in src]
            masses[n] = masses[n][src]

    most = prompt
    if prompt > budget:
        evict()
        most = budget
    for step in range(steps):
        if most >= budget + every:
            evict()
            most = budget
        q, kn, vn = rnd(N, Hq, d) * 1.5, rnd(N, Hkv, d), rnd(N, Hkv, d)
        out = c.attend(q.cuda(), kn.cuda(), vn.cuda())
        torch.cuda.synchronize()
        assert dd.dd_get_device_error() == dd.DD_OK
        most += 1
        for n in range(N):
            held[n].append((seen[n], CC.bits64(kn[n]), CC.bits64(vn[n])))
            seen[n] += 1
            m = len(held[n])
            assert int(c.lengths[n]) == m
            assert c.pos[n, :m].tolist() == [h[0] for h in held[n]]
            kk, vv = (np.stack([h[i] for h in held[n]])[None] for i in (1, 2))  # one page of m slots
            x = dict(q=q[n:n + 1], k=torch.tensor(kk), v=torch.tensor(vv), k_new=None, v_new=None,
                     table=torch.zeros(1, 1, dtype=torch.int32), max_len=m,
                     lengths=torch.tensor([m], dtype=torch.int32),
                     mass=torch.tensor(np.concatenate([masses[n], [0, 0, 0, 0]])[None].astype(np.float32)))
            ref = CC.attention_reference(x)
            got = dict(out=out[n:n + 1], lse=c.lse[n:n + 1], mass=torch.cat([c.mass[n:n + 1, :m].cpu(), torch.zeros(1, 3)], 1))
            CC.check_attention(x, got, ref, dtype)
            masses[n] = c.mass[n, :m].cpu().numpy()


@pytest.mark.parametrize("dtype,page,L", [(torch.bfloat16, 4, 10), (torch.float32, 3, 9), (torch.bfloat16, 16, 5),
                                          (torch.bfloat16, 1, 7)])
def test_beam_decode(dtype, page, L):
    layers, B, K, Hq, Hkv, d, V, steps = 2, 2, 4, 4, 2, 64, 50, 14
    gen = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(dtype)
    k, v = rnd(layers, B, L, Hkv, d), rnd(layers, B, L, Hkv, d)
    dec = BeamDecode(k.cuda(), v.cuda(), Hq, K, V, steps, page_size=page, eos=3)
    # every beam's own full history: per layer a list of rows, and its tokens
    hist = [[[(CC.bits64(k[l, n // K, j]), CC.bits64(v[l, n // K, j])) for j in range(L)]
             for l in range(layers)] for n in range(B * K)]
    toks = [[] for _ in range(B * K)]
    for t in range(steps):
        dec.begin()
        for l in range(layers):
            q, kn, vn = rnd(B * K, Hq, d), rnd(B * K, Hkv, d), rnd(B * K, Hkv, d)
            out = dec.attend(l, q.cuda(), kn.cuda(), vn.cuda())
            torch.cuda.synchronize()
            for n in range(B * K):
                hist[n][l].append((CC.bits64(kn[n]), CC.bits64(vn[n])))
                m = len(hist[n][l])
                kk, vv = (np.stack([h[i] for h in hist[n][l]])[None] for i in (0, 1))
                x = dict(q=q[n:n + 1], k=torch.tensor(kk), v=torch.tensor(vv), k_new=None, v_new=None, mass=None,
                         table=torch.zeros(1, 1, dtype=torch.int32), max_len=m,
                         lengths=torch.tensor([m], dtype=torch.int32))
                ref = CC.attention_reference(x)
                got = dict(out=out[n:n + 1], lse=torch.tensor(ref["lse"]))
                CC.check_attention(x, got, ref, dtype)
        logits = torch.randn(B, K, V, generator=gen) * 2
        wide = torch.zeros(B, K, 56)
        wide[..., :V] = logits
        score, done = dec.score.cpu().numpy(), dec.done.cpu().numpy()
        dec.advance(wide.cuda()[..., :V])
        torch.cuda.synchronize()
        assert dd.dd_get_device_error() == dd.DD_OK
        parent = []
        for b in range(B):
            p, tk, s, dn = OC.beam_select(logits[b].numpy().astype(np.float64), score[b], done[b], 3)
            assert dec.parent[b].tolist() == p.tolist() and dec.token[b].tolist() == tk.tolist(), t
            assert dec.done[b].tolist() == dn.tolist()
            parent.append(p)
        rows = OC.parents(np.array(parent), K)
        hist = [[list(hist[p][l]) for l in range(layers)] for p in rows]
        toks = [toks[p] + [int(dec.token.view(-1)[n])] for n, p in enumerate(rows)]
        assert dec.tokens.view(B * K, -1)[:, :t + 1].tolist() == toks
    with pytest.raises(ValueError):
        dec.begin()


def test_prompt_masses_from_the_verification_attention():
    """A prompt's keys, values and d_in come out of dd_dualview_attention as they are."""
    B, L, Hq, Hkv, d = 2, 96, 8, 4, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v = rnd(B, L, Hq, d), rnd(B, L, Hkv, d), rnd(B, L, Hkv, d)
    out, lse = torch.empty_like(q), torch.empty(B, Hq, L, device="cuda")
    d_in = torch.empty(B, L, device="cuda")
    every = torch.ones(B, L, dtype=torch.uint8, device="cuda")
    ws = torch.empty(dd.dd_dualview_attention_workspace_size(B, L, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    dd.dd_dualview_attention(q, k, v, None, None, None, every, None, out, lse, d_in, None, ws)
    c = BudgetedCache(B, Hq, Hkv, d, budget=32, page_size=16, sink=0, recent=0, prompt=L)
    c.fill(k, v, d_in)
    for b in range(B):
        want = OC.evict_one(d_in[b].cpu().numpy(), np.arange(L), 32, 0, 0)
        assert c.pos[b, :32].tolist() == want and int(c.lengths[b]) == 32
    # single-token attention over the whole prompt is the same attention
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    o, z = torch.empty(B, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hq, device="cuda")
    n = torch.full((B,), L, dtype=torch.int32, device="cuda")
    dd.dd_paged_attention(q[:, 5].contiguous(), dd.PagedCache(k, v, table), n, o, z)
    assert torch.allclose(o.float(), out[:, 5].float(), atol=2e-2)
    assert torch.allclose(z, lse[:, :, 5], atol=1e-3)


@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("page,L", [(1, 3), (2, 4), (3, 9), (16, 5)])
def test_beams_hold_their_own_histories(pattern, page, L):
    beams_hold_their_histories(pattern, page, L, "cuda")
    assert dd.dd_get_device_error() == dd.DD_OK
