"""dd_cache_evict against the oracle: everything it writes is exact."""
import numpy as np
import pytest
import torch

from oracle import cached as OC
from speculative_verification_cover_b200 import dd

pytestmark = pytest.mark.gpu


def _case(seed, N, page, Hkv, d, lengths, dtype=torch.bfloat16, ties=False, heads_first=False,
          spread=True):
    gen = torch.Generator().manual_seed(seed)
    most = max(max(lengths), 1)
    width = -(-most // page)
    pages = N * width + 1
    shape = (pages, Hkv, page, d) if heads_first else (pages, page, Hkv, d)
    k, v = (torch.randn(shape, generator=gen).to(dtype).cuda() for _ in range(2))
    if heads_first:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    table = torch.randperm(pages, generator=gen)[:N * width].view(N, width).to(torch.int32)
    mass = torch.rand(N, most + 2, generator=gen) if spread else torch.zeros(N, most + 2)
    if ties:
        mass = (mass * 3).round()
    pos = torch.zeros(N, most + 2, dtype=torch.int32)
    for n, length in enumerate(lengths):
        pos[n, :length] = torch.randperm(length, generator=gen).to(torch.int32)
    return k, v, table, mass, pos


def _run(seed, budget, sink, recent, **case):
    lengths = case["lengths"]
    N, page = case["N"], case["page"]
    k, v, table, mass, pos = _case(seed, **case)
    k0, v0 = k.clone(), v.clone()
    cache = dd.PagedCache(k, v, table.cuda())
    out = (torch.full_like(mass, -7.0).cuda(), torch.full_like(pos, -7).cuda(), torch.full_like(pos, -7).cuda())
    lens = torch.tensor(lengths, dtype=torch.int32).cuda()
    lens_out = torch.full_like(lens, -7)

    def call():
        dd.dd_cache_evict(cache, lens, mass.cuda(), pos.cuda(), budget, out[0], out[1], lens_out,
                          sink=sink, recent=recent, src=out[2], max_len=max(max(lengths), 1))
        torch.cuda.synchronize()
        assert dd.dd_get_device_error() == dd.DD_OK

    call()
    first = [t.clone() for t in (k, v, *out, lens_out)]
    mm, pp, ss = (t.cpu().numpy() for t in out)
    want_k, want_v = k0.clone(), v0.clone()
    for n, length in enumerate(lengths):
        src = OC.evict_one(mass[n, :length].numpy(), pos[n, :length].numpy(), budget, sink, recent)
        left = len(src)
        assert int(lens_out[n]) == left
        assert ss[n, :left].tolist() == src
        assert np.array_equal(mm[n, :left], mass[n].numpy()[src], equal_nan=True)
        assert np.array_equal(pp[n, :left], pos[n].numpy()[src])
        for t in (mm, pp, ss):  # behind the new length: as it was
            assert np.all(t[n, left:] == -7)
        t, j = torch.tensor(src, dtype=torch.long), torch.arange(left)
        row = table[n].long()
        for want, was in ((want_k, k0), (want_v, v0)):
            want[row[j // page].cuda(), (j % page).cuda()] = was[row[t // page].cuda(), (t % page).cuda()]
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    call()  # again on the same inputs: the same result
    for a, b in zip(first, (k, v, *out, lens_out)):
        assert torch.equal(a, b) or torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (31, 0, 0), (32, 4, 8),
                                                (33, 33, 0), (64, 0, 64), (64, 10, 54), (200, 4, 32)])
def test_budgets(budget, sink, recent, ties):
    _run(1, budget, sink, recent, N=5, page=16, Hkv=2, d=64, lengths=[200, 65, 1, 0, 199], ties=ties)


@pytest.mark.parametrize("page", [1, 3, 16, 100])
@pytest.mark.parametrize("dtype,d,Hkv", [(torch.bfloat16, 128, 8), (torch.float32, 128, 1),
                                         (torch.float32, 64, 3), (torch.bfloat16, 64, 1)])
def test_layouts(page, dtype, d, Hkv):
    for heads_first in (False, True):
        _run(2, 60, 2, 5, N=3, page=page, Hkv=Hkv, d=d, lengths=[61, 150, 77], dtype=dtype,
             heads_first=heads_first)


@pytest.mark.parametrize("length,budget", [(1025, 1024), (3001, 1024), (20000, 1), (20000, 19999),
                                           (70001, 30001), (100000, 64)])
def test_long(length, budget):
    _run(3, budget, 0, min(budget, 16) // 2, N=2, page=64, Hkv=1, d=64, lengths=[length, length // 2])
    _run(4, budget, 1, 0, N=1, page=64, Hkv=1, d=64, lengths=[length], ties=True)


def test_equal_masses_everywhere():
    _run(5, 700, 4, 32, N=2, page=16, Hkv=1, d=64, lengths=[2000, 701], spread=False)


def test_special_masses():
    inf, nan = float("inf"), float("nan")
    k, v, table, _, _ = _case(6, N=1, page=4, Hkv=1, d=64, lengths=[8])
    for m in ([nan, 0.0, -0.0, inf, -inf, nan, 1.0, -1.0], [nan] * 8, [-inf] * 8, [0.0, -0.0] * 4):
        for budget in (1, 3, 5, 7):
            mass = torch.tensor([m], device="cuda")
            pos = torch.arange(8, dtype=torch.int32, device="cuda")[None]
            mo, po, src = torch.zeros_like(mass), torch.zeros_like(pos), torch.zeros_like(pos)
            n = torch.tensor([8], dtype=torch.int32, device="cuda")
            dd.dd_cache_evict(dd.PagedCache(k, v, table.cuda()), n, mass, pos, budget, mo, po,
                              torch.zeros_like(n), src=src)
            assert src[0, :budget].tolist() == OC.evict_one(np.array(m), np.arange(8), budget, 0, 0), (m, budget)


def test_more_protected_than_the_budget_and_extreme_positions():
    k, v, table, _, _ = _case(7, N=1, page=4, Hkv=1, d=64, lengths=[8])
    big, low = 2 ** 31 - 1, -2 ** 31
    for p in ([0] * 8, [big] * 8, [low] * 8, [big, low, 0, 5, big, low, 3, 1]):
        mass = torch.rand(1, 8, generator=torch.Generator().manual_seed(1)).cuda()
        pos = torch.tensor([p], dtype=torch.int32, device="cuda")
        src = torch.zeros_like(pos)
        n = torch.tensor([8], dtype=torch.int32, device="cuda")
        dd.dd_cache_evict(dd.PagedCache(k, v, table.cuda()), n, mass, pos, 3, torch.zeros_like(mass),
                          torch.zeros_like(pos), torch.zeros_like(n), sink=1, recent=2, src=src)
        assert src[0, :3].tolist() == OC.evict_one(mass[0].cpu().numpy(), np.array(p, dtype=np.int64), 3, 1, 2), p


def test_holes_and_bad_values_move_nothing():
    k, v, table, mass, pos = _case(8, N=1, page=4, Hkv=1, d=64, lengths=[12])
    k0, v0 = k.clone(), v.clone()
    mass = torch.tensor([[0.0, 1, 0, 1, 1, 1, 1, 1, 9, 9, 9, 9]], device="cuda")
    pos = torch.arange(12, dtype=torch.int32, device="cuda")[None]
    out = (torch.zeros_like(mass), torch.zeros_like(pos))
    n, no = (torch.tensor([12], dtype=torch.int32, device="cuda") for _ in range(2))
    t = table.clone()
    t[0, 2] = -1                                     # the movers' page is a hole
    dd.dd_cache_evict(dd.PagedCache(k, v, t.cuda()), n, mass, pos, 8, *out, no)
    assert torch.equal(k, k0) and torch.equal(v, v0) and int(no) == 8
    assert dd.dd_get_device_error() == dd.DD_OK
    t[0, 2] = k.shape[0] + 5                         # or lies behind the pool
    dd.dd_cache_evict(dd.PagedCache(k, v, t.cuda()), n, mass, pos, 8, *out, no)
    assert torch.equal(k, k0) and torch.equal(v, v0)
    assert dd.dd_get_device_error() == dd.DD_ERR_BOUNDS
    n.fill_(400)                                     # a length beyond the rows is clamped
    dd.dd_cache_evict(dd.PagedCache(k, v, table.cuda()), n, mass, pos, 8, *out, no)
    assert int(no) == 8 and dd.dd_get_device_error() == dd.DD_ERR_BOUNDS
    n.fill_(-1)
    dd.dd_cache_evict(dd.PagedCache(k, v, table.cuda()), n, mass, pos, 8, *out, no)
    assert int(no) == 0 and dd.dd_get_device_error() == dd.DD_ERR_BOUNDS


@pytest.mark.parametrize("length,budget", [(290001, 100), (400000, 399000), (524288, 262144)])
def test_longest(length, budget):
    # keys that do not fit shared memory; the most movers there can be
    _run(20, budget, 3, 10, N=1, page=64, Hkv=1, d=64, lengths=[length])
    _run(21, budget, 0, 0, N=1, page=64, Hkv=1, d=64, lengths=[length], ties=True)


@pytest.mark.parametrize("lengths", [[2048, 2049, 100], [2049], [9000, 0, 1, 3000]])
def test_around_the_cluster_s_length(lengths):
    for budget in (1, 100, 2000, 2048):
        _run(22, budget, 1 if budget > 1 else 0, min(budget // 2, 64), N=len(lengths), page=16, Hkv=2, d=64,
             lengths=lengths)


def test_graph_replay_follows_lengths():
    for most in (600, 5000):
        k, v, table, mass, pos = _case(23, N=2, page=16, Hkv=1, d=64, lengths=[most, most])
        k0 = k.clone()
        cache, mass, pos = dd.PagedCache(k, v, table.cuda()), mass.cuda(), pos.cuda()
        lens = torch.tensor([most, most], dtype=torch.int32, device="cuda")
        mo, po, src, no = torch.zeros_like(mass), torch.zeros_like(pos), torch.zeros_like(pos), torch.zeros_like(lens)
        call = lambda: dd.dd_cache_evict(cache, lens, mass, pos, 256, mo, po, no, sink=2, recent=20, src=src)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        k.copy_(k0)
        lens.copy_(torch.tensor([most - 7, 200], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert no.tolist() == [256, 200]
        for n, length in enumerate(lens.tolist()):
            want = OC.evict_one(mass[n, :length].cpu().numpy(), pos[n, :length].cpu().numpy(), 256, 2, 20)
            assert src[n, :len(want)].tolist() == want


def test_refusals_of_the_binding():
    k, v, table, mass, pos = _case(24, N=2, page=16, Hkv=1, d=64, lengths=[60, 60])
    cache, mass, pos = dd.PagedCache(k, v, table.cuda()), mass.cuda(), pos.cuda()
    lens = torch.tensor([60, 60], dtype=torch.int32, device="cuda")

    def call(**over):
        a = dict(lengths=lens, mass=mass, pos=pos, budget=30, mass_out=torch.zeros_like(mass),
                 pos_out=torch.zeros_like(pos), lengths_out=torch.zeros_like(lens))
        a.update(over)
        dd.dd_cache_evict(cache, **a)

    call()
    for over in (dict(mass=mass.double()), dict(mass=mass[:1]), dict(mass=mass.cpu()), dict(pos=pos.long()),
                 dict(pos=pos[:, :-1]), dict(mass_out=mass[:, :10]), dict(lengths=lens.cpu()), dict(lengths=lens[:1]),
                 dict(src=pos.long()), dict(mass=mass.t().contiguous().t())):
        with pytest.raises((ValueError, TypeError)):
            call(**over)
    for over in (dict(budget=0), dict(sink=31), dict(mass_out=mass), dict(pos_out=pos), dict(lengths_out=lens),
                 dict(max_len=100), dict(recent=-1)):
        with pytest.raises(dd.DDError):
            call(**over)


def test_outputs_in_other_arguments_memory_are_refused():
    k, v, table, mass, pos = _case(30, N=2, page=16, Hkv=1, d=64, lengths=[60, 60])
    cache, mass, pos = dd.PagedCache(k, v, table.cuda()), mass.cuda(), pos.cuda()
    lens = torch.tensor([60, 60], dtype=torch.int32, device="cuda")
    mo, po = torch.zeros_like(mass), torch.zeros_like(pos)
    for over in (dict(src=pos), dict(src=po), dict(pos_out=mass.view(torch.int32)), dict(lengths_out=pos[0, 5:7])):
        a = dict(pos_out=po, lengths_out=torch.zeros_like(lens))
        a.update(over)
        with pytest.raises(dd.DDError):
            dd.dd_cache_evict(cache, lens, mass, pos, 30, mo, **a)
