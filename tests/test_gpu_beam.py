"""dd_beam_select, dd_beam_reorder and dd_paged_fork against the oracle.

Candidates are compared exactly. Scores of different beams can lie closer than the sums'
rounding: a log-sum of V fp32 exponentials is off by less than 2^-22 + V 2^-24 relative at
the very worst and, with errors of either sign, by about 2^-22; cases whose best K + 1
candidates of different beams lie within 4e-6 would be skipped, and none of these seeds has
one (asserted)."""
import numpy as np
import pytest
import torch

from oracle import cached as OC
from speculative_verification_cover_b200 import dd

pytestmark = pytest.mark.gpu
GAP = 4e-6


def _select(logits, score, done=None, eos=-1, **kw):
    B, K, V = logits.shape
    i = dict(dtype=torch.int32, device="cuda")
    parent, token = torch.full((B, K), -9, **i), torch.full((B, K), -9, **i)
    out = torch.full((B, K), 7.0, device="cuda")
    done_out = torch.full((B, K), 9, dtype=torch.uint8, device="cuda")
    dd.dd_beam_select(logits, score, parent, token, out, done=done, done_out=done_out, eos=eos, **kw)
    torch.cuda.synchronize()
    assert dd.dd_get_device_error() == dd.DD_OK
    return parent.cpu().numpy(), token.cpu().numpy(), out.cpu().numpy(), done_out.cpu().numpy()


def _check(logits, score, done=None, eos=-1, gaps=True):
    got = _select(logits, score, done, eos)
    x = logits.float().cpu().numpy()
    B, K, V = x.shape
    for b in range(B):
        dn = None if done is None else done[b].cpu().numpy()
        if gaps:
            best = OC.beam_candidates(x[b], score[b].cpu().numpy(), dn, eos, V, K + 1)
            for (s, i), (s2, i2) in zip(best, best[1:]):
                assert i // V == i2 // V or s2 - s > GAP
        parent, token, out, ended = OC.beam_select(x[b], score[b].cpu().numpy(), dn, eos)
        assert got[0][b].tolist() == parent.tolist(), b
        assert got[1][b].tolist() == token.tolist(), b
        assert got[3][b].tolist() == ended.tolist(), b
        fin = np.isfinite(out)
        assert np.array_equal(np.isneginf(got[2][b]), ~fin)
        # half a step of the value, and the log-sum's error
        assert np.all(np.abs(got[2][b][fin] - out[fin]) <= 2.0 ** -24 * np.abs(out[fin]) + 1e-6)
    return got


def _logits(seed, B, K, V, dtype, pad=0, std=3.0):
    gen = torch.Generator().manual_seed(seed)
    ld = -(-(V + pad) // 8) * 8
    x = (torch.randn(B, K, ld, generator=gen) * std).to(dtype)
    x[..., V:] = float("inf")  # columns behind the vocabulary are not candidates
    score = -torch.rand(B, K, generator=gen) * 4 - 10
    return x.cuda()[..., :V], score.cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (1, 4, 3), (2, 3, 7), (3, 1, 4097), (2, 5, 1000), (1, 64, 63),
                                   (2, 64, 9000), (4, 8, 32003), (1, 16, 126464), (2, 33, 8193)])
def test_shapes(dtype, B, K, V):
    x, score = _logits(1, B, K, V, dtype, pad=8)
    gen = torch.Generator().manual_seed(2)
    done = (torch.rand(B, K, generator=gen) < 0.2).to(torch.uint8).cuda()
    _check(x, score)
    _check(x, score, done, eos=V // 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_go_to_the_lowest_index(dtype):
    # equal logits in a beam: by index; equal beams: by beam
    for K, V in ((4, 10), (8, 20000), (64, 9000)):
        x = torch.zeros(2, K, -(-V // 8) * 8, dtype=dtype, device="cuda")[..., :V]
        _check(x, torch.zeros(2, K, device="cuda"), gaps=False)
        _check(x, torch.arange(2 * K, device="cuda").view(2, K).float(), gaps=False)
    x, _ = _logits(3, 1, 6, 5000, dtype)
    x = x[:, :1].round().expand(1, 6, 5000)
    wide = torch.empty(1, 6, 5000, dtype=dtype, device="cuda").copy_(x)
    _check(wide, torch.zeros(1, 6, device="cuda"), gaps=False)
    two = wide.clone()
    two[..., ::2] = -0.0
    two[..., 1::2] = 0.0
    _check(two, torch.zeros(1, 6, device="cuda"), gaps=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_thread_and_one_beam_hold_all_the_best(dtype):
    # every large logit within one vector's stride of threads; one beam far ahead
    x, score = _logits(4, 1, 64, 30000, dtype, std=1.0)
    x[0, :, 4096:4096 + 64] = torch.arange(64, device="cuda").to(dtype) + 20
    _check(x, score)
    score[0, 17] = 0.0
    _check(x, score)
    for stride in (256 * 8, 256 * 4):
        x[0, 17, 5::stride] = 60.0 + torch.arange(x[0, 17, 5::stride].numel(), device="cuda").to(dtype)
        _check(x, score)


def test_banned_and_empty():
    inf, nan = float("inf"), float("nan")
    x, score = _logits(5, 2, 4, 100, torch.float32, pad=4)
    x[0, 0] = -inf                     # a beam without candidates
    x[0, 1, 3:] = -inf                 # three tokens left
    x[0, 2, ::2] = nan
    x[1] = -inf                        # a request without candidates
    _check(x, score)
    score[0, 3] = -inf                 # an empty slot
    score[0, 2] = nan
    _check(x, score)
    done = torch.zeros(2, 4, dtype=torch.uint8, device="cuda")
    done[1, 2] = done[0, 3] = 1
    _check(x, score, done, eos=0)
    _check(x, score, done, eos=-1)
    done.fill_(1)
    _check(x, score, done, eos=99)


def test_first_step_starts_from_one_beam():
    x, _ = _logits(6, 3, 8, 5000, torch.bfloat16)
    score = torch.full((3, 8), float("-inf"), device="cuda")
    score[:, 0] = 0.0
    got = _check(x, score)
    assert np.all(got[0] == 0)


def test_other_stream_and_graph():
    x, score = _logits(7, 4, 8, 20000, torch.bfloat16)
    want = _select(x, score)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _select(x, score, stream=side)
    for a, b in zip(want, got):
        assert np.array_equal(a, b)
    i = dict(dtype=torch.int32, device="cuda")
    parent, token, out = torch.zeros(4, 8, **i), torch.zeros(4, 8, **i), torch.zeros(4, 8, device="cuda")
    ws = torch.empty(dd.dd_beam_select_workspace_size(4, 8, 20000, torch.bfloat16), dtype=torch.uint8,
                     device="cuda")
    call = lambda: dd.dd_beam_select(x, score, parent, token, out, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    y, s2 = _logits(8, 4, 8, 20000, torch.bfloat16)
    x.copy_(y)
    score.copy_(s2)
    graph.replay()
    torch.cuda.synchronize()
    want = _select(y, s2)
    assert np.array_equal(parent.cpu().numpy(), want[0]) and np.array_equal(token.cpu().numpy(), want[1])


@pytest.mark.parametrize("shape,dtype", [((1,), torch.uint8), ((7,), torch.uint8), ((3,), torch.int32),
                                         ((5, 4), torch.float32), ((129, 257), torch.bfloat16),
                                         ((100000,), torch.int32)])
def test_reorder(shape, dtype):
    B, K = 3, 5
    gen = torch.Generator().manual_seed(9)
    parent = torch.randint(-1, K + 1, (B, K), generator=gen).to(torch.int32)
    states = [torch.randint(0, 100, (B, K, *shape), generator=gen).to(dtype).cuda(),
              torch.randint(0, 100, (B * K, *shape), generator=gen).to(dtype).cuda()]
    outs = [torch.full_like(s, 101) for s in states]
    dd.dd_beam_reorder(parent.cuda(), list(zip(states, outs)))
    rows = torch.tensor(OC.parents(parent.numpy(), K)).cuda()
    for s, o in zip(states, outs):
        assert torch.equal(o.view(B * K, -1), s.view(B * K, -1)[rows])


@pytest.mark.parametrize("layers,page,Hkv,d,dtype", [(1, 16, 8, 128, torch.bfloat16), (3, 5, 1, 64, torch.float32),
                                                     (2, 1, 2, 64, torch.bfloat16), (1, 128, 4, 128, torch.float32)])
def test_fork(layers, page, Hkv, d, dtype):
    B, K = 3, 4
    N = B * K
    rng = np.random.default_rng(10)
    width = 4
    cap = width * page
    lengths = rng.integers(0, cap + 1, N)
    lengths[:4] = [0, page, cap, min(cap, page + 1)]
    pages = N * width + N + 3
    ids = rng.permutation(pages)
    table = ids[:N * width].reshape(N, width).copy()
    table[5, :] = -1                                   # holes stay holes
    fresh = ids[N * width:N * width + N]
    parent = rng.integers(-1, K, (B, K))
    k, v = (torch.randn(layers, pages, page, Hkv, d).to(dtype) for _ in range(2))
    kw, vw, tw = k.float().numpy().copy(), v.float().numpy().copy(), np.full((N, width), -7)
    lw = OC.fork(parent, K, table, lengths, fresh, kw, vw, tw)
    t = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    kg, vg, out, lout = k.cuda(), v.cuda(), t(np.full((N, width), -7)), t(np.zeros(N))
    dd.dd_paged_fork(dd.PagedCache(kg, vg, t(table)), t(parent), t(lengths), t(fresh), out, lout)
    torch.cuda.synchronize()
    assert dd.dd_get_device_error() == dd.DD_OK
    assert np.array_equal(out.cpu().numpy(), tw) and np.array_equal(lout.cpu().numpy(), lw)
    assert np.array_equal(kg.float().cpu().numpy(), kw) and np.array_equal(vg.float().cpu().numpy(), vw)


def test_fork_records_bad_pages_and_lengths():
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    k = torch.randn(6, 4, 1, 64, device="cuda")
    v = torch.randn_like(k)
    k0 = k.clone()
    table, out, lout = t([[0, 1], [2, 3]]), t([[-7, -7], [-7, -7]]), t([0, 0])
    cache = dd.PagedCache(k, v, table)
    dd.dd_paged_fork(cache, t([[1, 0]]), t([5, 6]), t([6, -1]), out, lout)  # both fresh pages are bad
    assert dd.dd_get_device_error() == dd.DD_ERR_BOUNDS
    assert torch.equal(k, k0) and out.tolist() == [[2, -1], [0, -1]] and lout.tolist() == [6, 5]
    dd.dd_paged_fork(cache, t([[0, 1]]), t([100, -3]), t([4, 5]), out, lout)
    assert dd.dd_get_device_error() == dd.DD_ERR_BOUNDS
    assert torch.equal(k, k0) and out.tolist() == [[0, 1], [5, -1]] and lout.tolist() == [8, 0]


def test_more_pieces_and_entries_than_are_held_on_chip():
    x, score = _logits(20, 1, 64, 152064, torch.bfloat16)
    _check(x, score)
    x, score = _logits(21, 1, 48, 152064, torch.float32)
    _check(x, score)
    _check(torch.zeros_like(x), torch.zeros_like(score), gaps=False)


def test_values_that_are_not_finite():
    inf, nan = float("inf"), float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        x, score = _logits(22, 2, 4, 20000, dtype)
        x[0, 0, 7] = inf                   # no candidate, not in the sum
        x[0, 1, ::3] = nan
        x[0, 2, :] = inf
        x[1, 3, 16384:] = -inf
        x[1, 2, 100:9000] = inf
        score[1, 0] = inf                  # empty slots
        score[1, 1] = nan
        got = _check(x, score)
        assert 0 not in got[0][1] and 1 not in got[0][1] and 2 not in got[0][0]


def test_scores_of_any_size():
    # far below zero (a long hypothesis), and far apart
    x, score = _logits(23, 2, 8, 5000, torch.bfloat16)
    wide = score * 1e4
    _check(x, wide)
    _check(x, score * 1e30, gaps=False)


def test_refusals_of_the_binding():
    x, score = _logits(24, 2, 4, 1000, torch.bfloat16)
    i = dict(dtype=torch.int32, device="cuda")

    def call(**over):
        a = dict(logits=x, score=score, parent=torch.zeros(2, 4, **i), token=torch.zeros(2, 4, **i),
                 score_out=torch.zeros(2, 4, device="cuda"))
        a.update(over)
        dd.dd_beam_select(**a)

    call()
    for over in (dict(logits=x.half()), dict(logits=x.cpu()), dict(logits=x[:, :3]), dict(logits=x[..., ::2]), dict(logits=x[0]),
                 dict(logits=x.transpose(0, 1)), dict(score=score.double()), dict(score=score[:1]), dict(parent=torch.zeros(2, 4)),
                 dict(done=torch.zeros(2, 4, dtype=torch.bool, device="cuda")), dict(token=torch.zeros(2, 4, dtype=torch.int32)),
                 dict(workspace=torch.zeros(10))):
        with pytest.raises((ValueError, TypeError)):
            call(**over)
    for over in (dict(score_out=score), dict(eos=1000), dict(eos=-2), dict(logits=x[..., :999], eos=999),
                 dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(dd.DDError):
            call(**over)
    parent = torch.zeros(2, 4, **i)
    s = torch.zeros(8, 5, device="cuda")
    for pair in ((s, s), (s, s[:, :4]), (s, s.int()), (s.cpu(), s), (torch.zeros(16, 5, device="cuda")[:8], torch.zeros(7, 5, device="cuda")),
                 (s.t().contiguous().t(), s.clone())):
        with pytest.raises((ValueError, TypeError)):
            dd.dd_beam_reorder(parent, [pair])
    big = torch.zeros(12, 5, device="cuda")
    with pytest.raises(ValueError):                     # one within the other's memory
        dd.dd_beam_reorder(parent, [(big[:8], big[4:])])
    with pytest.raises(dd.DDError):
        dd.dd_beam_reorder(parent, [])
    with pytest.raises(dd.DDError):
        dd.dd_beam_reorder(parent, [(s, s.clone())] * 9)


def _check_range(logits, score, done=None, eos=-1):
    """_check for scores that fp32 may not hold: what lies below its range is -inf."""
    got = _select(logits, score, done, eos)
    x = logits.float().cpu().numpy()
    for b in range(x.shape[0]):
        dn = None if done is None else done[b].cpu().numpy()
        parent, token, out, ended = OC.beam_select(x[b], score[b].cpu().numpy(), dn, eos)
        assert got[0][b].tolist() == parent.tolist(), b
        assert got[1][b].tolist() == token.tolist(), b
        assert got[3][b].tolist() == ended.tolist(), b
        with np.errstate(over="ignore"):
            want = out.astype(np.float32).astype(np.float64)
        fin = np.isfinite(want)
        assert np.array_equal(got[2][b][~fin], want[~fin])
        assert np.all(np.abs(got[2][b][fin] - out[fin]) <= 2.0 ** -24 * np.abs(out[fin]) + 1e-6)


def _masked(x, where, mask):
    """x with the logits of a pattern at the mask's value: eight vectors of 16 bytes, every 256th
    of a piece of 32 KB, are one thread's segment; 32 such segments a warp's."""
    V, per = x.shape[-1], 16 // x.element_size()
    i = torch.arange(V, device=x.device)
    thread, piece = i // per % 256, i // (per * 2048)
    hit = {"segment": (thread == 7) & (piece == 0), "warp": (thread // 32 == 1) & (piece == 0), "piece": piece == 0,
           "all but one": i != V // 3, "all but twenty": i % (V // 20) != 0, "row": i >= 0}[where]
    return torch.where(hit, mask, x.float()).to(x.dtype)


MASKS = [lambda f: f.min, lambda f: -f.max / 2, lambda f: -1e38, lambda f: -1e30, lambda f: -1e20, lambda f: -1e10,
         lambda f: -3e9, lambda f: -65504.0]


@pytest.mark.parametrize("mask", range(len(MASKS)))
@pytest.mark.parametrize("where", ["segment", "warp", "piece", "all but one", "all but twenty", "row"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_finite_masks(dtype, where, mask):
    """Tokens banned by a large negative finite value, in one beam and in all of them."""
    value = MASKS[mask](torch.finfo(dtype))
    for V in (1000, 20000):
        wide, score = _logits(30, 2, 5, V, dtype)
        x = wide.clone()
        x[:, 2] = _masked(x[:, 2], where, value)
        _check_range(x, score)
        x = _masked(wide, where, value)
        _check_range(x, score)
        done = torch.zeros(2, 5, dtype=torch.uint8, device="cuda")
        done[:, 3] = 1
        _check_range(x, score, done, eos=5)
        # no logit of the row left, or some
        x[0, 1] = float("-inf")
        x[1, 4, ::2] = float("-inf")
        _check_range(x, score)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_finite_logits(dtype):
    f = torch.finfo(dtype)
    for best in (1e5, 1e10, 1e30, f.max / 2, f.max):
        for V in (1000, 20000):
            x, score = _logits(31, 2, 4, V, dtype)
            x[:, torch.arange(4), torch.arange(4) * 7 + 3] = torch.tensor(best, dtype=dtype, device="cuda")
            _check_range(x, score)          # each beam's best; the rest far behind
            x[0, 1] = f.min
            x[1, :, V // 2:] = f.min
            _check_range(x, score)
            score[:, 1:] = float("-inf")    # one beam: its other tokens are all that follows
            _check_range(x, score)
    # a whole row at the largest value, one of it at the lowest: every distance overflows
    x, score = _logits(32, 1, 3, 9000, dtype)
    x[0, 0], x[0, 1], x[0, 2] = f.max, f.min, f.max
    x[0, 2, 1::2] = f.min
    _check_range(x, score)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 15, 1001, 8191, 8193, 16385, 20001])
def test_a_contiguous_row_that_ends_its_storage(dtype, V):
    """One beam's logits, unpadded: the last, partly filled 16 bytes are the row's own alone."""
    gen = torch.Generator().manual_seed(33)
    x = torch.randn(1, 1, V, generator=gen).to(dtype).cuda()
    x[..., -1] = 9.0
    got = _check(x, torch.zeros(1, 1, device="cuda"))
    assert int(got[1][0, 0]) == V - 1
    # what lies behind a row of a wider buffer is not read: the largest there is, right behind
    wide = torch.full((2, 3, -(-(V + 1) // 8) * 8), torch.finfo(dtype).max, dtype=dtype, device="cuda")
    wide[..., :V] = torch.randn(2, 3, V, generator=gen).to(dtype).cuda()
    _check(wide[..., :V], torch.tensor([[0.0, -1.0, -2.5], [-0.3, -1.1, -2.0]], device="cuda"))
