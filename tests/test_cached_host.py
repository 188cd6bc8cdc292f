"""Host side of the cached operators' binding, without a GPU: the checks of CPU tensors (in
the place of a device's) up to the library's call, which is recorded and not made."""
import ctypes
import importlib.metadata
import os

import pytest
import torch

from speculative_verification_cover_b200 import build, dd


@pytest.fixture
def calls(monkeypatch):
    build.build()
    made = []
    monkeypatch.setattr(dd, "_gpu", lambda t, name: -1)  # what the compiled checks call the CPU
    monkeypatch.setattr(dd, "_call", lambda name, gpu, stream, *args: made.append((name, args)))
    return made


def _cache(N=2, pages=8, page=16, Hkv=2, d=64, width=8):
    k, v = (torch.zeros(pages, page, Hkv, d) for _ in range(2))
    return dd.PagedCache(k, v, torch.zeros(N, width, dtype=torch.int32))


@pytest.mark.parametrize("B", [1, 2, 3])
def test_masses_narrower_than_max_len_are_refused(calls, B):
    """Masses may be columns of a wider buffer: a max_len above their width would have the
    call write what lies behind them."""
    cache = _cache(N=B)
    q, n = torch.zeros(B, 4, 64), torch.zeros(B, dtype=torch.int32)
    wide = torch.zeros(B, 128)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    call = lambda **kw: dd.dd_paged_attention(q, cache, n, torch.zeros_like(q), workspace=ws, **kw)
    call(mass_out=wide[:, :50], max_len=50)
    call(mass=wide[:, :50], mass_out=wide[:, :50], max_len=7)
    call(mass_out=wide[:, :50])
    assert [c[1][9] for c in calls] == [50, 7, 50]  # max_len as the library gets it
    for kw in (dict(mass_out=wide[:, :50], max_len=51), dict(mass_out=wide[:, :50], max_len=128),
               dict(mass=wide[:, 50:60], mass_out=wide[:, :10], max_len=11)):
        with pytest.raises(dd.DDError):
            call(**kw)
    assert len(calls) == 3


def test_the_binding_s_part_is_rebuilt_for_its_header_python_and_torch(monkeypatch):
    """It has the header's signatures compiled in, and reads torch's tensors."""
    path = build.args_path()
    build.build()
    assert os.path.exists(path) and build.up_to_date(path)
    times = {path: 1.0, build.HEADER: 2.0}
    with monkeypatch.context() as m:
        m.setattr(os.path, "getmtime", lambda p: times.get(p, 0.0))
        assert not build.up_to_date(path)
        times[build.HEADER] = 1.0
        assert build.up_to_date(path)
        times[build.ARGS_SOURCE] = 2.0
        assert not build.up_to_date(path)
    with monkeypatch.context() as m:
        m.setattr(importlib.metadata, "version", lambda name: "0.0")
        assert build.args_path() != path and not build.up_to_date(build.args_path())
        m.setattr(dd, "_host", None)
        with pytest.raises(ImportError, match="torch0.0"):
            dd._load_host()


@pytest.mark.parametrize("missing", ["compiler", "headers", "torch"])
def test_libraries_build_without_the_binding_s_part(monkeypatch, tmp_path, missing):
    """The verification step and the C ABI need nvcc alone."""
    build.build()
    part = str(tmp_path / "part.so")
    monkeypatch.setattr(build, "args_path", lambda: part)
    if missing == "torch":
        def command(out):
            raise ImportError("No module named 'torch'")
        monkeypatch.setattr(build, "_args_command", command)
    else:
        monkeypatch.setenv("CXX", "false" if missing == "headers" else str(tmp_path / "no_such_compiler"))
    for old in (False, True):
        if old:  # one that is older than its sources does not stay
            open(part, "w").close()
            os.utime(part, (0, 0))
        with pytest.warns(UserWarning, match="not built"):
            assert build.build() == build.OUT
        assert not os.path.exists(part)
    monkeypatch.setattr(dd, "_host", None)
    with pytest.raises(ImportError, match="is missing: build it"):
        dd._load_host()


# Addresses that are never dereferenced: every call below is refused before any device work.
IN, OUT = 0x10000000, 0x20000000


def _table(**over):
    a = dict(k=0x1000000, v=0x2000000, layer_stride=0, page_stride=4096, token_stride=256, head_stride=64, layers=1,
             n_pages=10, page_size=16, Hkv=4, d=64, dtype=1, page_table=0x30000000, table_stride=8, max_pages=8)
    a.update(over)
    return ctypes.byref(dd._PagedCache(**a))


def _spread(names, start):
    """Addresses of a megabyte each."""
    return {n: start + (i << 20) for i, n in enumerate(names)}


def _evict(**over):
    a = _spread(("lengths", "mass", "pos"), IN) | _spread(("mass_out", "pos_out", "src", "lengths_out"), OUT)
    a.update(over)
    return dd.lib().dd_cache_evict(_table(), a["lengths"], 2, 100, 50, 4, 8, a["mass"], a["pos"], 100, a["mass_out"],
                                   a["pos_out"], a["src"], a["lengths_out"], None)


def _select(**over):
    a = _spread(("x", "score", "done"), IN) | _spread(("parent", "token", "score_out", "done_out", "ws"), OUT)
    a.update(over)
    return dd.lib().dd_beam_select(a["x"], 1, 2, 4, 100, 104, a["score"], a["done"], -1, a["parent"], a["token"],
                                   a["score_out"], a["done_out"], a["ws"], 1 << 20, None)


def _fork(**over):
    a = _spread(("parent", "lengths", "fresh"), IN) | _spread(("table_out", "lengths_out"), OUT)
    a.update(over)
    return dd.lib().dd_paged_fork(_table(), a["parent"], 2, 4, a["lengths"], a["fresh"], a["table_out"], 8,
                                  a["lengths_out"], None)


def _attend(**over):
    a = _spread(("q", "kn", "vn", "lengths", "mass"), IN) | _spread(("out", "lse", "mass_out", "ws"), OUT)
    a.update(over)
    return dd.lib().dd_paged_attention(a["q"], 512, a["kn"], a["vn"], 256, _table(), a["lengths"], 2, 8, 100, 0.0,
                                       a["out"], a["lse"], a["mass"], a["mass_out"], 100, a["ws"], 1 << 40, None)


def _reorder(pairs, parent=IN, stride=16):
    rows = (dd._RowState * len(pairs))(*[dd._RowState(s, d, 8, stride, stride) for s, d in pairs])
    return dd.lib().dd_beam_reorder(parent, 2, 4, rows, len(pairs), None)


def test_outputs_in_the_memory_of_inputs_or_other_outputs_are_refused():
    """CTAs of a call read its inputs while others write: src_out as pos_in would have clusters
    choose different slots, lengths_out as fresh would send rows to another beam's page."""
    build.build()
    a = _spread(("lengths", "mass", "pos"), IN) | _spread(("mass_out", "pos_out", "src", "lengths_out"), OUT)
    table = 0x30000000
    row = 100 * 4
    evict = [dict(src=a["pos"]), dict(src=a["mass"]), dict(src=a["pos_out"]), dict(src=a["mass_out"]),
             dict(src=a["pos"] + row + 99 * 4), dict(pos_out=a["mass"]), dict(mass_out=a["pos"]), dict(mass_out=a["pos_out"]),
             dict(mass_out=a["mass"] - 49 * 4), dict(pos_out=a["pos"] + 4), dict(lengths_out=a["lengths"] + 4),
             dict(lengths_out=a["pos"] + 4), dict(lengths_out=a["mass_out"]), dict(lengths_out=table + 60),
             dict(src=table - row - 196)]
    for over in evict:
        assert _evict(**over) == dd.DD_ERR_INVALID_ARG, over
    a = _spread(("x", "score", "done"), IN) | _spread(("parent", "token", "score_out", "done_out", "ws"), OUT)
    for over in (dict(token=a["parent"]), dict(score_out=a["parent"] + 28), dict(done_out=a["token"] + 31),
                 dict(parent=a["score"]), dict(parent=a["done"]), dict(token=a["x"] + 7 * 208 + 199), dict(score_out=a["score"] - 28),
                 dict(done_out=a["done"] + 7), dict(ws=a["parent"]), dict(ws=a["x"]), dict(done_out=a["ws"] + 5)):
        assert _select(**over) == dd.DD_ERR_INVALID_ARG, over
    a = _spread(("parent", "lengths", "fresh"), IN) | _spread(("table_out", "lengths_out"), OUT)
    for over in (dict(lengths_out=a["fresh"]), dict(lengths_out=a["parent"]), dict(lengths_out=a["lengths"] + 28),
                 dict(table_out=a["fresh"]), dict(table_out=a["parent"] + 16), dict(table_out=table + 7 * 32),
                 dict(table_out=table - 32), dict(lengths_out=a["table_out"] + 200), dict(lengths_out=table)):
        assert _fork(**over) == dd.DD_ERR_INVALID_ARG, over
    a = _spread(("q", "kn", "vn", "lengths", "mass"), IN) | _spread(("out", "lse", "mass_out", "ws"), OUT)
    for over in (dict(out=a["q"] + 16), dict(out=a["kn"]), dict(out=a["vn"] - 2032), dict(lse=a["lengths"]), dict(lse=a["out"]),
                 dict(mass_out=a["mass"] + 4), dict(mass_out=a["mass"] - row), dict(mass_out=a["lse"]), dict(ws=a["q"]),
                 dict(lse=table + 60), dict(ws=a["mass_out"] + 256)):
        assert _attend(**over) == dd.DD_ERR_INVALID_ARG, over
    # rows 16 bytes apart, 8 used
    for pairs, parent in (([(IN, OUT), (OUT, OUT + 4096)], 1), ([(IN, OUT), (IN, OUT)], 1), ([(IN, OUT), (IN + 8, OUT + 4)], 1),
                          ([(IN, OUT)], OUT + 7 * 16 + 4), ([(IN, IN + 7 * 16 + 7)], 1), ([(IN, IN - 16)], 1),
                          ([(IN, OUT), (OUT + 8, IN + 7 * 16)], 1)):
        assert _reorder(pairs, parent) == dd.DD_ERR_INVALID_ARG, pairs
