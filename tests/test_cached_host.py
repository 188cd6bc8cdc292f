"""Host side of the cached operators' binding, without a GPU: the checks of CPU tensors (in
the place of a device's) up to the library's call, which is recorded and not made."""
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
