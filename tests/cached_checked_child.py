"""Child process of test_gpu_cached_checked.py (not collected by pytest): runs the cached
operators on the library the binding loads -- the checked build when the parent sets
DD_CHECK_BOUNDS=1 -- and saves every output to the path given as argv[1]."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from speculative_verification_cover_b200 import dd  # noqa: E402
from tests import cached_cases as CC  # noqa: E402


def attention():
    out = {}
    for name, case in (
            ("ranges", dict(B=3, Hq=28, Hkv=4, d=128, page=16, lengths=[900, 1, 333], mass=True)),
            ("heads16", dict(B=2, Hq=20, Hkv=2, d=128, page=5, lengths=[700, 65], mass=True)),
            ("cluster", dict(B=1, Hq=8, Hkv=2, d=64, page=16, lengths=[400])),
            ("whole", dict(B=60, Hq=8, Hkv=4, d=64, page=16, lengths=list(range(0, 480, 8)))),
            ("fp32", dict(B=3, Hq=8, Hkv=1, d=128, page=16, lengths=[900, 1, 333], mass=True, dtype=torch.float32))):
        g = CC.on_gpu(CC.make_attention(1, **case))
        got = CC.run_attention(g)
        got.update(k=g["k"].nan_to_num(), v=g["v"].nan_to_num(), status=torch.tensor(dd.dd_get_device_error()))
        out[name] = {k: v.cpu() for k, v in got.items() if v is not None}
    return out


def evict():
    out = {}
    gen = torch.Generator(device="cuda").manual_seed(2)
    for n, budget in ((1000, 700), (6000, 1000), (20000, 19000)):
        for ties in (False, True):
            k = torch.randn(n // 16 + 1, 16, 2, 64, device="cuda", generator=gen).bfloat16()
            v = torch.randn(k.shape, device="cuda", generator=gen).bfloat16()
            table = torch.randperm(k.shape[0], device="cuda", generator=gen).int()[None]
            mass = torch.rand(1, n, device="cuda", generator=gen)
            mass = (mass * 4).round() if ties else mass
            pos = torch.randperm(n, device="cuda", generator=gen).int()[None]
            mo, po, src = torch.zeros_like(mass), torch.zeros_like(pos), torch.zeros_like(pos)
            lens = torch.tensor([n], dtype=torch.int32, device="cuda")
            dd.dd_cache_evict(dd.PagedCache(k, v, table), lens, mass, pos, budget, mo, po, torch.zeros_like(lens),
                              sink=4, recent=32, src=src)
            out[f"{n}_{ties}"] = {"k": k.cpu(), "v": v.cpu(), "mass": mo.cpu(), "pos": po.cpu(), "src": src.cpu(),
                                  "status": torch.tensor(dd.dd_get_device_error())}
    return out


def beam():
    out = {}
    gen = torch.Generator(device="cuda").manual_seed(3)
    for name, x in (("spread", torch.randn(2, 8, 20000, device="cuda", generator=gen)),
                    ("equal", torch.zeros(2, 64, 9000, device="cuda"))):
        B, K, _ = x.shape
        i = dict(dtype=torch.int32, device="cuda")
        parent, token, score = torch.zeros(B, K, **i), torch.zeros(B, K, **i), torch.zeros(B, K, device="cuda")
        dd.dd_beam_select(x, torch.zeros(B, K, device="cuda"), parent, token, score)
        out[name] = {"parent": parent.cpu(), "token": token.cpu(), "score": score.cpu(),
                     "status": torch.tensor(dd.dd_get_device_error())}
    return out


if __name__ == "__main__":
    torch.save({"checked": dd.dd_bounds_checked(), "attention": attention(), "evict": evict(), "beam": beam()},
               sys.argv[1])
