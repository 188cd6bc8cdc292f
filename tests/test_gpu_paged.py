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


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (7, 1), (16, 1), (34, 1), (32, 16)])
@pytest.mark.parametrize("lengths,max_len", [([1], 1), ([64], 64), ([33], 64), ([65], 65), ([200], 300),
                                             ([511], 512), ([0], 512), ([512, 0, 17], 512),
                                             ([300, 5, 0, 64, 129] * 8, 300)])
def test_short_sequences_without_masses(dtype, d, Hq, Hkv, lengths, max_len):
    # one launch: a cluster for each sequence-head, or whole ones to a CTA
    B = len(lengths)
    holes = [(b, 0) for b, n in enumerate(lengths) if n > 40 and b % 3 == 0]
    _check(20, B=B, Hq=Hq, Hkv=Hkv, d=d, page=16, lengths=lengths, max_len=max_len, dtype=dtype, holes=holes)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_whole_sequences_of_a_large_batch(dtype):
    gen = np.random.default_rng(21)
    lengths = gen.integers(0, 400, 100).tolist()
    lengths[:3] = [0, 0, 512]
    lengths[-1] = 0
    _check(21, B=100, Hq=12, Hkv=4, d=64, page=24, lengths=lengths, max_len=512, dtype=dtype)


def test_a_length_out_of_range_appends_nothing():
    for mass in (False, True):
        x = CC.make_attention(22, B=2, Hq=4, Hkv=2, d=64, page=16, lengths=[64, 30], mass=mass)
        g = CC.on_gpu(x)
        k0 = g["k"].clone()
        g["lengths"][0] = 65
        CC.run_attention(g)
        assert dd.dd_get_device_error() == dd.DD_ERR_BOUNDS
        page, row = int(x["table"][0, 3]), 15
        assert torch.equal(g["k"][page, row], k0[page, row])
        page, row = int(x["table"][1, 1]), 29 - 16
        assert torch.equal(g["k"][page, row].cpu(), x["k_new"][1])


def test_an_append_into_a_hole_is_dropped():
    x = CC.make_attention(23, B=1, Hq=4, Hkv=2, d=64, page=16, lengths=[40], mass=True, holes=[(0, 2)])
    _check(23, B=1, Hq=4, Hkv=2, d=64, page=16, lengths=[40], mass=True, holes=[(0, 2)])
    _check(23, B=1, Hq=4, Hkv=2, d=64, page=16, lengths=[33], mass=False, holes=[(0, 2)])
    assert int(x["table"][0, 2]) == -1


@pytest.mark.parametrize("mass", [False, True])
def test_two_calls_at_once(mass):
    xs = [CC.make_attention(30 + i, B=6, Hq=16, Hkv=4, d=128, page=16, lengths=[900, 20, 700, 1, 350, 40],
                            mass=mass) for i in range(2)]
    gs = [CC.on_gpu(x) for x in xs]
    want = [CC.run_attention(g) for g in gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    n = dd.dd_paged_attention_workspace_size(6, 16, 4, 128, 900, mass)
    spaces = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in gs]
    torch.cuda.synchronize()
    got = []
    for rep in range(20):
        got = [CC.run_attention(g, stream=s, workspace=w) for g, s, w in zip(gs, streams, spaces)]
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for key in a:
            assert a[key] is None or torch.equal(a[key], b[key]), key


def test_strided_rows():
    # masses as columns of a wider table, new tokens as slices of a fused projection
    x = CC.make_attention(40, B=3, Hq=8, Hkv=4, d=64, page=16, lengths=[100, 640, 7], mass=True)
    g = CC.on_gpu(x)
    B, M = g["mass"].shape
    wide = torch.full((2, B, M + 5), 3.0, device="cuda")
    wide[0, :, :M] = g["mass"]
    fused = torch.zeros(B, 3 * 4 * 64, dtype=BF16, device="cuda")
    fused[:, 256:512] = g["k_new"].view(B, -1)
    fused[:, 512:] = g["v_new"].view(B, -1)
    out, lse = torch.empty(B, 8, 64, dtype=BF16, device="cuda"), torch.empty(B, 8, device="cuda")
    wide[1, :, :M] = g["mass"]
    dd.dd_paged_attention(g["q"], dd.PagedCache(g["k"], g["v"], g["table"]), g["lengths"], out, lse,
                          k_new=fused[:, 256:512].view(B, 4, 64), v_new=fused[:, 512:].view(B, 4, 64),
                          mass=wide[0, :, :M], mass_out=wide[1, :, :M], max_len=x["max_len"])
    torch.cuda.synchronize()
    CC.check_attention(x, dict(out=out, lse=lse, mass=wide[1, :, :M]), CC.attention_reference(x), BF16)
    assert torch.all(wide[:, :, M:] == 3.0)


def test_refusals_of_the_binding():
    x = CC.make_attention(41, B=2, Hq=4, Hkv=2, d=64, page=16, lengths=[20, 30], mass=True)
    g = CC.on_gpu(x)
    cache = dd.PagedCache(g["k"], g["v"], g["table"])
    out, lse = torch.empty_like(g["q"]), torch.empty(2, 4, device="cuda")

    def call(**over):
        a = dict(q=g["q"], cache=cache, lengths=g["lengths"], out=out, lse=lse, k_new=g["k_new"],
                 v_new=g["v_new"], mass=g["mass"], mass_out=torch.zeros_like(g["mass"]))
        a.update(over)
        dd.dd_paged_attention(a.pop("q"), a.pop("cache"), a.pop("lengths"), a.pop("out"), **a)

    call()
    bad = [dict(q=g["q"].float()), dict(q=g["q"].cpu()), dict(q=g["q"][:1]), dict(q=g["q"][:, :3]), dict(q=g["q"][..., :32]),
           dict(q=g["q"].transpose(0, 1).contiguous().transpose(0, 1)), dict(lengths=g["lengths"].long()),
           dict(lengths=g["lengths"][:1]), dict(lengths=g["lengths"].cpu()), dict(out=out.float()), dict(out=out[:, :2]),
           dict(lse=lse.double()), dict(lse=lse[:, :2]), dict(k_new=None), dict(v_new=None), dict(k_new=g["k_new"].cpu()),
           dict(k_new=g["k_new"][:, :1]), dict(mass_out=None), dict(mass=g["mass"][:, :-1]), dict(mass=g["mass"].double()),
           dict(workspace=torch.empty(1 << 20, dtype=torch.uint8)), dict(mass_out=torch.zeros(2, 60, device="cuda")[:, ::2])]
    for over in bad:
        with pytest.raises((ValueError, TypeError)):
            call(**over)
    for over in (dict(max_len=10 ** 6), dict(max_len=0), dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(dd.DDError):
            call(**over)
    for k, v, t in ((g["k"], g["v"].float(), g["table"]), (g["k"], g["v"][:, :8], g["table"]), (g["k"], g["v"], g["table"].long()),
                    (g["k"], g["v"], g["table"].cpu()), (g["k"], g["v"], g["table"][0]), (g["k"][..., ::2], g["v"][..., ::2], g["table"]),
                    (g["k"].half(), g["v"].half(), g["table"])):
        with pytest.raises((ValueError, TypeError)):
            dd.PagedCache(k, v, t)
    call()
    torch.cuda.synchronize()
    assert dd.dd_get_device_error() == dd.DD_OK


def test_pools_that_share_memory_are_read_only():
    """One key head expanded to all heads (or one tensor as keys and values) can be attended
    to; what would write it is refused."""
    x = CC.make_attention(21, B=2, Hq=4, Hkv=2, d=64, page=8, lengths=[9, 20], append=False)
    x["k"], x["v"] = (t[:, :, :1].expand(-1, -1, 2, -1) for t in (x["k"], x["v"]))
    g = {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}
    g["k"], g["v"] = (x[n][:, :, :1].contiguous().cuda().expand(-1, -1, 2, -1) for n in ("k", "v"))
    assert g["k"].stride(2) == 0
    got = CC.run_attention(g)
    torch.cuda.synchronize()
    CC.check_attention(x, got, CC.attention_reference(x), BF16)
    cache = dd.PagedCache(g["k"], g["v"], g["table"])
    new = torch.zeros(2, 2, 64, dtype=BF16, device="cuda")
    out, parent = torch.empty_like(g["q"]), torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    n, f = g["lengths"], torch.zeros(2, 20, device="cuda")
    i = torch.zeros(2, 20, dtype=torch.int32, device="cuda")
    k = torch.zeros(8, 8, 2, 64, dtype=BF16, device="cuda")
    for c in (cache, dd.PagedCache(k, k, g["table"])):
        assert c.read_only
        with pytest.raises(ValueError, match="only be read"):
            dd.dd_paged_attention(g["q"], c, n, out, k_new=new, v_new=new)
        with pytest.raises(ValueError, match="only be read"):
            dd.dd_cache_evict(c, n, f, i, 5, f.clone(), i.clone(), n.clone())
        with pytest.raises(ValueError, match="only be read"):
            dd.dd_paged_fork(c, parent, n, n.clone(), torch.empty_like(g["table"]), n.clone())


def test_empty_batches_are_refused():
    i = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(dd.DDError):
        dd.dd_beam_reorder(i, [(torch.zeros(0, 3, device="cuda"), torch.zeros(0, 3, device="cuda"))])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,Hq,Hkv,lengths", [
    (1, 256, 32, [12]), (40, 80, 8, [1, 4, 0, 3]), (160, 4, 1, [128, 1, 77, 0]), (80, 6, 2, [120, 512, 300, 5]),
    (64, 8, 8, [200, 512]), (130, 16, 4, [33, 64, 2])])
def test_masses_of_short_sequences(dtype, B, Hq, Hkv, lengths):
    """Whole sequence-heads, with the masses from their own log-sums: more heads than a warp
    takes at once, empty sequences, pages that are holes, all rounds of CTAs."""
    lengths = (lengths * B)[:B]
    holes = [(b, 0) for b in range(0, B, 7) if lengths[b] > 8]
    _check(24, B=B, Hq=Hq, Hkv=Hkv, d=64, page=8, lengths=lengths, dtype=dtype, mass=True, holes=holes)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths", [[700, 31, 512, 0], [50, 64, 1, 0], [300], [200, 5, 0, 64, 129] * 12])
@pytest.mark.parametrize("mass", [False, True])
def test_outputs_beside_and_in_place_of_inputs(dtype, lengths, mass):
    """The output in the queries' place, and masses in columns between each other's: the same bits."""
    x = CC.make_attention(50, B=len(lengths), Hq=40, Hkv=4, d=64, page=16, lengths=lengths, mass=mass, dtype=dtype)
    want = CC.run_attention(CC.on_gpu(x))
    g = CC.on_gpu(x)
    B, M = len(lengths), x["max_len"] + 3
    both = torch.full((B, 2, M), 7.0, device="cuda")
    kw = {}
    if mass:
        both[:, 0] = g["mass"]
        both[:, 1] = g["mass"]
        kw = dict(mass=both[:, 0], mass_out=both[:, 1])
    dd.dd_paged_attention(g["q"], dd.PagedCache(g["k"], g["v"], g["table"]), g["lengths"], g["q"], k_new=g["k_new"],
                          v_new=g["v_new"], max_len=x["max_len"], **kw)
    torch.cuda.synchronize()
    assert dd.dd_get_device_error() == dd.DD_OK
    assert torch.equal(g["q"], want["out"])
    if mass:
        assert torch.equal(both[:, 1], want["mass"]) and torch.equal(both[:, 0], g["mass"])


def test_overlapping_outputs_are_refused():
    x = CC.make_attention(51, B=2, Hq=4, Hkv=2, d=64, page=16, lengths=[20, 30], mass=True)
    g = CC.on_gpu(x)
    cache = dd.PagedCache(g["k"], g["v"], g["table"])
    buf = torch.zeros(4096, device="cuda")
    q = buf[:512].view(BF16)[:512].view(2, 4, 64)
    for kw in (dict(out=buf.view(BF16)[8:520].view(2, 4, 64)), dict(out=g["k_new"].new_zeros(2, 4, 64), lse=buf[:8].view(2, 4)),
               dict(out=torch.zeros_like(q), mass=buf[600:666].view(2, 33), mass_out=buf[601:667].view(2, 33))):
        with pytest.raises(dd.DDError):
            dd.dd_paged_attention(q, cache, g["lengths"], kw.pop("out"), max_len=30, **kw)
