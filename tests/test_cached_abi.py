"""The cached-decoding entry points refuse bad arguments on the host, before any device
work (CPU only; no compute call is made)."""
import ctypes

import pytest
import torch

from speculative_verification_cover_b200 import build, dd

P = ctypes.c_void_p
FAKE = 0x10000          # never dereferenced: validation fails first
OTHER = 0x20000
ODD = 0x10008
WS = 0x100000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dd.lib()


def _cache(**over):
    a = dict(k=FAKE, v=FAKE, layer_stride=0, page_stride=4096, token_stride=256, head_stride=64, layers=1,
             n_pages=10, page_size=16, Hkv=4, d=64, dtype=1, page_table=FAKE, table_stride=8, max_pages=8)
    a.update(over)
    return ctypes.byref(dd._PagedCache(**a))


BAD_CACHES = [dict(k=None), dict(v=None), dict(page_table=None), dict(dtype=5), dict(n_pages=0), dict(page_size=0),
              dict(Hkv=0), dict(max_pages=0), dict(d=0), dict(k=ODD), dict(v=ODD), dict(token_stride=65),
              dict(head_stride=-64), dict(page_stride=4097), dict(table_stride=7), dict(layers=0)]


def _attend(lib, cache=None, **over):
    a = dict(q=FAKE, qs=512, kn=None, vn=None, ns=256, lengths=FAKE, B=2, Hq=8, max_len=100, scale=0.0, out=FAKE,
             lse=None, mi=None, mo=None, ms=0, ws=WS, wsb=1 << 40)
    a.update(over)
    return lib.dd_paged_attention(a["q"], a["qs"], a["kn"], a["vn"], a["ns"], _cache(**(cache or {})), a["lengths"],
                                  a["B"], a["Hq"], a["max_len"], a["scale"], a["out"], a["lse"], a["mi"], a["mo"],
                                  a["ms"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_every_call_checks_its_cache(lib, bad):
    assert _attend(lib, cache=bad) == dd.DD_ERR_INVALID_ARG
    assert _evict(lib, cache=bad) == dd.DD_ERR_INVALID_ARG
    assert _fork(lib, cache=bad) == dd.DD_ERR_INVALID_ARG


def test_paged_attention_validation(lib):
    inv, uns = dd.DD_ERR_INVALID_ARG, dd.DD_ERR_UNSUPPORTED
    for bad in (dict(q=None), dict(lengths=None), dict(out=None), dict(B=0), dict(Hq=0), dict(Hq=6), dict(max_len=0),
                dict(max_len=129), dict(kn=FAKE), dict(vn=FAKE), dict(q=ODD), dict(out=ODD), dict(kn=FAKE, vn=ODD),
                dict(qs=504), dict(qs=513), dict(kn=FAKE, vn=FAKE, ns=248), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(mi=FAKE), dict(mo=FAKE, ms=99), dict(ws=None), dict(ws=WS + 64),
                dict(wsb=100)):
        assert _attend(lib, **bad) == inv, bad
    assert _attend(lib, cache=dict(layers=2)) == inv
    assert lib.dd_paged_attention(FAKE, 512, None, None, 0, None, FAKE, 1, 8, 10, 0.0, FAKE, None, None, None, 0,
                                  WS, 1 << 40, None) == inv
    assert _attend(lib, cache=dict(d=96)) == uns
    assert _attend(lib, B=4097) == uns
    assert _attend(lib, Hq=8196, qs=8196 * 64) == uns
    big = dict(max_pages=1 << 27, table_stride=1 << 27)
    assert _attend(lib, cache=big, max_len=(1 << 31) - 1, B=4096, qs=512) == uns
    need = dd.dd_paged_attention_workspace_size(2, 8, 4, 64, 100, True)
    assert _attend(lib, mo=FAKE, ms=100, wsb=need - 1) == inv
    assert need >= 2 * 8 * 100 * 4 and need % 256 == 0
    assert dd.dd_paged_attention_workspace_size(2, 8, 4, 64, 100) < need
    for bad in ((0, 8, 4, 64, 100), (2, 7, 4, 64, 100), (2, 8, 4, 64, 0), (2, 8, 0, 64, 9)):
        assert dd.dd_paged_attention_workspace_size(*bad) == 0


def _evict(lib, cache=None, **over):
    a = dict(lengths=FAKE, N=2, max_len=100, budget=50, sink=4, recent=8, mi=FAKE, pi=FAKE, stride=100, mo=OTHER,
             po=OTHER, src=None, lo=OTHER)
    a.update(over)
    return lib.dd_cache_evict(_cache(**(cache or {})), a["lengths"], a["N"], a["max_len"], a["budget"], a["sink"],
                              a["recent"], a["mi"], a["pi"], a["stride"], a["mo"], a["po"], a["src"], a["lo"], None)


def test_evict_validation(lib):
    inv, uns = dd.DD_ERR_INVALID_ARG, dd.DD_ERR_UNSUPPORTED
    for bad in (dict(lengths=None), dict(mi=None), dict(pi=None), dict(mo=None), dict(po=None), dict(lo=None),
                dict(N=0), dict(max_len=0), dict(max_len=129), dict(budget=0), dict(sink=-1), dict(recent=-1),
                dict(sink=43), dict(recent=47), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(stride=99),
                dict(mo=FAKE), dict(po=FAKE), dict(lo=FAKE)):
        assert _evict(lib, **bad) == inv, bad
    assert _evict(lib, cache=dict(layers=2)) == inv
    assert _evict(lib, N=65536) == uns
    big = dict(max_pages=1 << 16, table_stride=1 << 16)
    assert _evict(lib, cache=big, max_len=524289, stride=524289) == uns


def _select(lib, **over):
    a = dict(x=FAKE, dtype=1, B=2, K=4, V=100, ld=104, s=FAKE, done=None, eos=-1, p=OTHER, t=OTHER, so=OTHER, do=None,
             ws=WS, wsb=1 << 40)
    a.update(over)
    return lib.dd_beam_select(a["x"], a["dtype"], a["B"], a["K"], a["V"], a["ld"], a["s"], a["done"], a["eos"], a["p"],
                              a["t"], a["so"], a["do"], a["ws"], a["wsb"], None)


def test_beam_select_validation(lib):
    inv, uns = dd.DD_ERR_INVALID_ARG, dd.DD_ERR_UNSUPPORTED
    for bad in (dict(x=None), dict(s=None), dict(p=None), dict(t=None), dict(so=None), dict(dtype=3), dict(B=0),
                dict(K=0), dict(V=0), dict(ld=99), dict(ld=100), dict(eos=-2), dict(eos=100), dict(x=ODD),
                dict(so=FAKE), dict(done=FAKE, do=FAKE), dict(ws=None), dict(ws=WS + 8), dict(wsb=64)):
        assert _select(lib, **bad) == inv, bad
    assert _select(lib, K=65) == uns
    assert _select(lib, V=(1 << 23) + 1, ld=1 << 24) == uns
    assert _select(lib, B=1 << 20) == uns
    n = dd.dd_beam_select_workspace_size(2, 4, 100, torch.bfloat16)
    assert n > 0 and _select(lib, wsb=n - 1) == inv
    assert dd.dd_beam_select_workspace_size(2, 65, 100, torch.bfloat16) == 0
    assert dd.dd_beam_select_workspace_size(0, 4, 100, torch.bfloat16) == 0


def test_reorder_validation(lib):
    inv, uns = dd.DD_ERR_INVALID_ARG, dd.DD_ERR_UNSUPPORTED

    def call(n=1, B=2, K=4, parent=FAKE, **over):
        s = dict(src=FAKE, dst=OTHER, row_bytes=8, src_stride=8, dst_stride=8)
        s.update(over)
        arr = (dd._RowState * max(n, 1))(*[dd._RowState(**s)] * max(n, 1))
        return lib.dd_beam_reorder(parent, B, K, arr, n, None)

    for bad in (dict(parent=None), dict(n=0), dict(B=0), dict(K=0), dict(src=None), dict(dst=None), dict(dst=FAKE),
                dict(row_bytes=0), dict(src_stride=7), dict(dst_stride=7)):
        assert call(**bad) == inv, bad
    assert lib.dd_beam_reorder(FAKE, 2, 4, None, 1, None) == inv
    assert call(n=9) == uns and call(B=1 << 20) == uns


def _fork(lib, cache=None, **over):
    a = dict(parent=FAKE, B=2, K=4, lengths=FAKE, fresh=FAKE, to=OTHER, stride=8, lo=OTHER)
    a.update(over)
    return lib.dd_paged_fork(_cache(**(cache or {})), a["parent"], a["B"], a["K"], a["lengths"], a["fresh"], a["to"],
                             a["stride"], a["lo"], None)


def test_fork_validation(lib):
    for bad in (dict(parent=None), dict(lengths=None), dict(fresh=None), dict(to=None), dict(lo=None), dict(B=0),
                dict(K=0), dict(stride=7), dict(to=FAKE), dict(lo=FAKE)):
        assert _fork(lib, **bad) == dd.DD_ERR_INVALID_ARG, bad
    assert _fork(lib, B=16384) == dd.DD_ERR_UNSUPPORTED
    assert _fork(lib, cache=dict(d=32)) == dd.DD_ERR_UNSUPPORTED


def test_binding_refuses_cpu_tensors():
    k, t = torch.zeros(2, 4, 1, 64), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        dd.PagedCache(k, k, t)
    with pytest.raises(ValueError):
        dd.dd_beam_select(torch.zeros(1, 2, 8), *[None] * 4)
    with pytest.raises(ValueError):
        dd.dd_beam_reorder(torch.zeros(1, 2, dtype=torch.int32), [])
    with pytest.raises(TypeError):
        dd.dd_beam_select([[1.0]], *[None] * 4)


@pytest.mark.parametrize("n", [1, 2, 3, 5, 7, 16, 24, 48, 100, 127, 128, 129, 1000, 65537, 2 ** 30 + 1, 2 ** 31 - 1])
def test_page_division_is_exact(n):
    """The multiplication that divides slots by the page size, in the kernels' arithmetic."""
    l = (n - 1).bit_length()
    m = (1 << (31 + l)) // n + 1
    assert m < 1 << 33
    for x in {0, 1, n - 1, n, n + 1, 2 * n - 1, 2 * n, 2 ** 31 - 1, 2 ** 31 - 2, (2 ** 31 - 1) // n * n,
              (2 ** 31 - 1) // n * n - 1, 2 ** 30, 12345}:
        if 0 <= x < 2 ** 31:
            assert x * m < 1 << 64 and (x * m) >> (31 + l) == x // n, x


@pytest.mark.parametrize("shape,stride,shared", [
    ((3, 4, 2, 64), (512, 128, 64, 1), False), ((3, 4, 2, 64), (512, 64, 256, 1), False),
    ((3, 4, 2, 64), (4096, 128, 64, 1), False), ((1, 4, 1, 64), (0, 64, 0, 1), False),
    ((3, 4, 2, 64), (0, 128, 64, 1), True), ((3, 4, 2, 64), (512, 128, 0, 1), True),
    ((3, 4, 2, 64), (256, 128, 64, 1), True), ((3, 4, 2, 64), (512, 64, 64, 1), True)])
def test_pools_whose_elements_share_memory(shape, stride, shared):
    assert dd._overlaps(shape, stride) is shared


def test_compiled_argument_checks(lib):
    """The binding's compiled checks (gpu -1 stands for the CPU here): addresses and strides,
    and an error that says what is wrong."""
    f32, cpu = torch.float32, -1
    t = torch.zeros(3, 4, 5)
    wide = torch.zeros(3, 32)
    assert dd._arg(t, "t", f32, (3, 4, 5), cpu) == t.data_ptr()
    assert dd._arg(torch.nn.Parameter(t), "t", f32, t.shape, cpu) == t.data_ptr()
    assert dd._rows(t, "t", f32, t.shape, cpu) == (t.data_ptr(), 20)
    assert dd._rows(wide[:, 2:7], "w", f32, (3, 5), cpu) == (wide.data_ptr() + 8, 32)
    assert dd._rows(wide[:, :20].unflatten(1, (4, 5)), "w", f32, (3, 4, 5), cpu) == (wide.data_ptr(), 32)
    assert dd._rows(wide[:1, 2:7], "w", f32, (1, 5), cpu)[0] == wide.data_ptr() + 8
    assert dd._arg(t[:0], "t", f32, (0, 4, 5), cpu) == 0
    with pytest.raises(TypeError, match="name_of_it: expected a torch.Tensor"):
        dd._arg([1.0], "name_of_it", f32, (1,), cpu)
    with pytest.raises(TypeError):
        dd._arg(None, "t", f32, (1,), cpu)
    for bad in ((torch.int32, (3, 4, 5)), (f32, (3, 4)), (f32, (3, 4, 6)), (f32, (3, 4, 5, 1)), (f32, ())):
        with pytest.raises(ValueError, match="must be torch"):
            dd._arg(t, "t", *bad, cpu)
        with pytest.raises(ValueError, match="must be torch"):
            dd._rows(t, "t", *bad, cpu)
    with pytest.raises(ValueError, match="cuda:0"):
        dd._arg(t, "t", f32, t.shape, 0)
    for view in (t.transpose(0, 1), t[:, ::2], t[..., :3]):
        for check in (dd._arg, dd._rows):
            with pytest.raises(ValueError, match="must be contiguous"):
                check(view, "t", f32, view.shape, cpu)
    with pytest.raises(ValueError, match="must be contiguous"):
        dd._arg(wide[:, 2:7], "w", f32, (3, 5), cpu)
    assert dd._workspace(wide, cpu) == (wide.data_ptr(), 3 * 32 * 4)
    for bad, error in ((wide[:, :4], ValueError), (b"ws", TypeError)):
        with pytest.raises(error):
            dd._workspace(bad, cpu)
    with pytest.raises(ValueError):
        dd._workspace(wide, 0)


def test_compiled_calls_check_their_arguments(lib):
    host = dd._host or dd._load_host()
    assert host.dd_cache_evict(None, None, 0, 0, 1, 0, 0, None, None, 0, *[None] * 5) == dd.DD_ERR_INVALID_ARG
    assert host.dd_beam_reorder(FAKE, 2, 4, [], None) == dd.DD_ERR_INVALID_ARG
    assert host.dd_beam_reorder(FAKE, 2, 4, [FAKE, OTHER, 8] * 9, None) == dd.DD_ERR_UNSUPPORTED
    assert host.dd_beam_reorder(FAKE, 2, 4, [FAKE, OTHER, 8, OTHER, OTHER, 8], None) == dd.DD_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        host.dd_cache_evict(None)
    with pytest.raises(TypeError):
        host.dd_beam_reorder(FAKE, 2, 4, (), None)
    with pytest.raises(OverflowError):
        host.dd_beam_reorder(FAKE, 2 ** 31, 4, [], None)
    with pytest.raises(TypeError):
        host.dd_beam_reorder(FAKE, 2, "4", [], None)
