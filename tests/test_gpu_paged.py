"""dd_paged_attention against the fp64 oracle (tolerances: tests/cached_cases.py)."""
import numpy as np
import pytest
import torch

from speculative_verification_cover_b200 import dd
from tests import cached_cases as CC

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _check(seed, kw=None, **case):
    x = CC.make_attention(seed, **case)
    g = CC.on_gpu(x)
    got = CC.run_attention(g, **(kw or {}))
    torch.cuda.synchronize()
    assert dd.dd_get_device_error() == dd.DD_OK
    ref = CC.attention_reference(x, scale=(kw or {}).get("softmax_scale"))
    CC.check_attention(x, got, ref, x["q"].dtype)
    # the cache: the appended slots are the new token's bits, everything else is as it was
    for key in ("k", "v"):
        want = ref[key]
        assert np.array_equal(CC.bits64(g[key]), want, equal_nan=True), key
    return x, got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (8, 4), (6, 2), (28, 4), (16, 2), (20, 2),
                                    (16, 1), (34, 1), (80, 8)])
def test_head_layouts(dtype, d, Hq, Hkv):
    _check(1, B=3, Hq=Hq, Hkv=Hkv, d=d, page=16, lengths=[1, 150, 33], dtype=dtype, mass=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [1, 2, 3, 5, 7, 16, 24, 48, 64, 100, 1000])
def test_page_sizes(dtype, page):
    _check(2, B=4, Hq=4, Hkv=2, d=64, page=page, lengths=[63, 64, 65, 130], dtype=dtype, mass=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 5003])
def test_lengths(dtype, n):
    _check(3, B=2, Hq=4, Hkv=2, d=128, page=16, lengths=[n, max(1, n // 3)], dtype=dtype, mass=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_empty_sequences_and_holes(dtype):
    # sequences without slots between others; one whose every page is a hole; holes inside
    # a tile, at both ends and over whole tiles
    _check(4, B=6, Hq=4, Hkv=2, d=64, page=8, lengths=[0, 40, 0, 20, 300, 0], dtype=dtype, mass=True,
           holes=[(1, 1), (1, 4), (3, 0), (3, 1), (3, 2), (4, 0)] + [(4, i) for i in range(8, 25)])
    _check(5, B=1, Hq=2, Hkv=2, d=64, page=8, lengths=[0], dtype=dtype, mass=True)


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("mass", [False, True])
def test_options(append, mass):
    _check(6, B=3, Hq=8, Hkv=4, d=128, page=32, lengths=[700, 31, 512], append=append, mass=mass,
           max_len=900)
    # pools stored heads first, q as a slice of wider rows, a scale of the caller's
    _check(7, B=3, Hq=8, Hkv=4, d=128, page=32, lengths=[70, 310, 512], append=append, mass=mass,
           heads_first=True, q_pad=64, kw=dict(softmax_scale=0.03))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_ragged_sequences(dtype):
    gen = np.random.default_rng(8)
    lengths = (2.0 ** gen.uniform(0, 9, 150)).astype(int).tolist()
    lengths[17] = 0
    _check(8, B=150, Hq=8, Hkv=4, d=64, page=16, lengths=lengths, dtype=dtype, mass=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_scores(dtype):
    # scores of hundreds: one slot takes all the weight, the rest underflow
    x, got = _check(9, B=2, Hq=4, Hkv=2, d=64, page=16, lengths=[200, 77], dtype=dtype, mass=True,
                    q_scale=200.0)
    assert float(got["lse"].max()) > 500


def test_runs_repeat_bit_for_bit_and_accumulate_in_place():
    x = CC.make_attention(10, B=5, Hq=28, Hkv=4, d=128, page=16, lengths=[900, 3, 411, 64, 1025], mass=True)
    g = CC.on_gpu(x)
    a, b = CC.run_attention(g), CC.run_attention(g)
    for key in a:
        assert torch.equal(a[key], b[key]), key
    # in place: the same sums
    cache = dd.PagedCache(g["k"], g["v"], g["table"])
    out, mass = torch.empty_like(a["out"]), g["mass"].clone()
    dd.dd_paged_attention(g["q"], cache, g["lengths"], out, k_new=g["k_new"], v_new=g["v_new"],
                          mass=mass, mass_out=mass, max_len=g["max_len"])
    assert torch.equal(mass, a["mass"]) and torch.equal(out, a["out"])
    # max_len sizes the launch, not the result beyond rounding; no masses before: zero
    zero = torch.zeros_like(mass)
    dd.dd_paged_attention(g["q"], cache, g["lengths"], out, k_new=g["k_new"], v_new=g["v_new"],
                          mass_out=zero)
    sums = [float(zero[b, :n].sum()) for b, n in enumerate(x["lengths"].tolist())]
    assert np.allclose(sums, 1.0, atol=1e-5)


def test_offsets_beyond_32_bits():
    # a pool of more than 2^32 bytes whose used pages lie at both ends
    Hkv, d, page = 8, 128, 64
    pages = (1 << 32) // (page * Hkv * d * 2) + 40
    k = torch.zeros(pages, page, Hkv, d, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    x = CC.make_attention(11, B=2, Hq=16, Hkv=Hkv, d=d, page=page, lengths=[100, 190], mass=True)
    small = x["k"].shape[0]
    where = torch.tensor([pages - 1 - i if i % 2 else i for i in range(small)], device="cuda")
    k[where], v[where] = x["k"].cuda(), x["v"].cuda()
    g = CC.on_gpu(x)
    g["k"], g["v"] = k, v
    g["table"] = where.to(torch.int32)[g["table"].long()]
    got = CC.run_attention(g)
    torch.cuda.synchronize()
    assert dd.dd_get_device_error() == dd.DD_OK
    ref = CC.attention_reference(x)
    CC.check_attention(x, got, ref, BF16)
    assert np.array_equal(CC.bits64(k[where]), ref["k"], equal_nan=True)


def test_bad_pages_and_lengths_are_recorded_not_read():
    x = CC.make_attention(12, B=3, Hq=4, Hkv=2, d=64, page=16, lengths=[50, 40, 64], mass=True, append=False)
    g = CC.on_gpu(x)
    g["table"][0, 1] = x["k"].shape[0]          # behind the pool: counts as a hole
    x["table"][0, 1] = -1
    got = CC.run_attention(g)
    assert dd.dd_get_device_error() == dd.DD_ERR_BOUNDS
    CC.check_attention(x, got, CC.attention_reference(x), BF16)
    # lengths outside [0, max_len] are clamped
    g = CC.on_gpu(x)
    g["lengths"][1], g["lengths"][2] = -5, 1000
    x["lengths"][1] = 0
    got = CC.run_attention(g)
    assert dd.dd_get_device_error() == dd.DD_ERR_BOUNDS
    CC.check_attention(x, got, CC.attention_reference(x), BF16)
    assert dd.dd_get_device_error() == dd.DD_OK


def test_other_stream_workspace_and_graph_replay():
    x = CC.make_attention(13, B=4, Hq=32, Hkv=8, d=128, page=16, lengths=[700, 1, 90, 255], mass=True,
                          max_len=1024)
    g = CC.on_gpu(x)
    want = CC.run_attention(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = CC.run_attention(g, stream=side)      # its workspace is allocated for that stream
    torch.cuda.current_stream().wait_stream(side)
    for key in want:
        assert torch.equal(got[key], want[key]), key
    # a captured call follows lengths, tables and values that change between replays
    cache = dd.PagedCache(g["k"], g["v"], g["table"])
    out, lse, mass = torch.empty_like(want["out"]), torch.empty_like(want["lse"]), g["mass"].clone()
    ws = torch.empty(dd.dd_paged_attention_workspace_size(4, 32, 8, 128, 1024, True), dtype=torch.uint8,
                     device="cuda")
    call = lambda: dd.dd_paged_attention(g["q"], cache, g["lengths"], out, lse, k_new=g["k_new"],
                                         v_new=g["v_new"], mass=g["mass"], mass_out=mass,
                                         max_len=1024, workspace=ws)
    call()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    y = CC.make_attention(14, B=4, Hq=32, Hkv=8, d=128, page=16, lengths=[3, 0, 980, 0], mass=True,
                          max_len=1024)
    for key in ("q", "table", "lengths", "k_new", "v_new", "mass"):
        g[key].copy_(y[key])
    pages = y["k"].shape[0]
    assert pages <= g["k"].shape[0]
    g["k"][:pages].copy_(y["k"])
    g["v"][:pages].copy_(y["v"])
    mass.copy_(y["mass"])
    graph.replay()
    torch.cuda.synchronize()
    CC.check_attention(y, dict(out=out, lse=lse, mass=mass), CC.attention_reference(y), BF16)
    assert dd.dd_get_device_error() == dd.DD_OK


def test_beams_read_shared_pages():
    # three sequences over the same full page, each with an open page of its own
    x = CC.make_attention(15, B=3, Hq=4, Hkv=2, d=64, page=16, lengths=[20, 25, 17], mass=True)
    x["table"][1, 0] = x["table"][2, 0] = x["table"][0, 0]
    g = CC.on_gpu(x)
    got = CC.run_attention(g)
    torch.cuda.synchronize()
    CC.check_attention(x, got, CC.attention_reference(x), BF16)
