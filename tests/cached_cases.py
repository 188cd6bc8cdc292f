"""Inputs and tolerances of the cached-decoding tests.

Tolerances, from the arithmetic (half a step of a type is finfo.eps / 2):
  score  a dot product of d terms in fp32, scaled: at most (d + 4) half steps of the sum of
         its terms' magnitudes, and another half step per unit for the change of base
  p      relative error 2 x the score's error (numerator and normaliser) plus the
         exponential's 2^-22 and a half step for each of the n terms of the normaliser
  out    p's relative error, n half steps for its own sum and 2^-16 for weights carried as
         two bf16 terms, times sum p |v|; and half a step of the output's type
  lse    the score's error, n half steps, half a step of its value
  mass   p's relative error times p, summed over heads; half a step of the running value
         for the sum over heads and the addition
Weights below 2^-126, the smallest normal fp32 number, may be flushed to zero: a slot's mass
loses at most 2^-126, an output n 2^-126 max |v| < 2^-112 for the n and v here.
"""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24


def bits64(t):
    """Exact fp64 values of a bf16 / fp32 tensor."""
    return t.detach().float().cpu().numpy().astype(np.float64)


def make_attention(seed, B, Hq, Hkv, d, page, lengths, dtype=torch.bfloat16, holes=(), append=True,
                   mass=False, max_len=None, heads_first=False, q_pad=0, q_scale=1.5):
    """A call's tensors on the CPU. holes: (sequence, page) pairs dropped from the tables;
    slots nobody may read hold NaN."""
    gen = torch.Generator().manual_seed(seed)
    lengths = torch.tensor(lengths, dtype=torch.int32)
    max_len = int(max(1, lengths.max())) if max_len is None else max_len
    width = -(-max_len // page)
    counts = ((lengths + page - 1) // page).tolist()
    ids = torch.randperm(sum(counts) + 2, generator=gen).to(torch.int32)
    pages = len(ids)
    table = torch.full((B, width), int(ids[-1]), dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        at += n
    shape = (pages, Hkv, page, d) if heads_first else (pages, page, Hkv, d)
    pools = []
    for _ in range(2):
        x = torch.full(shape, float("nan"), dtype=dtype)
        x = x.transpose(1, 2) if heads_first else x
        for b, n in enumerate(lengths.tolist()):
            j = torch.arange(n)
            x[table[b].long()[j // page], j % page] = torch.randn(n, Hkv, d, generator=gen).to(dtype)
        pools.append(x)
    for b, p in holes:
        table[b, p] = -1
    rows = torch.randn(B, Hq * d + q_pad, generator=gen).mul_(q_scale).to(dtype)
    x = dict(q=rows[:, :Hq * d].view(B, Hq, d), k=pools[0], v=pools[1], table=table, lengths=lengths,
             max_len=max_len)
    x["k_new"], x["v_new"] = ((torch.randn(B, Hkv, d, generator=gen).to(dtype) for _ in range(2))
                              if append else (None, None))
    x["mass"] = torch.rand(B, max_len + 3, generator=gen) if mass else None
    return x


def on_gpu(x, device="cuda"):
    """The same tensors on the GPU, strides kept."""
    out = {}
    for key, t in x.items():
        if isinstance(t, torch.Tensor):
            g = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=device)
            out[key] = g.copy_(t)
        else:
            out[key] = t
    return out


def attention_reference(x, scale=None):
    """fp64 outputs and the tolerances of each (out without its own rounding)."""
    from oracle import cached as OC
    q, k, v = bits64(x["q"]), bits64(x["k"]), bits64(x["v"])
    table, lengths = x["table"].numpy(), x["lengths"].numpy()
    kn, vn = (None if x[n] is None else bits64(x[n]) for n in ("k_new", "v_new"))
    B, Hq, d = q.shape
    page, Hkv = k.shape[1], k.shape[2]
    M = x["max_len"] + 3
    before = np.zeros((B, M)) if x["mass"] is None else bits64(x["mass"])
    out, lse, mass = OC.paged_attention(q, k, v, table, lengths, kn, vn, before, scale)
    sc = 1.0 / np.sqrt(d) if scale is None else scale
    t_out, t_lse, t_mass = np.zeros_like(out), np.zeros_like(lse), np.zeros_like(mass)
    for b in range(B):
        slots = OC.held_slots(table[b], int(lengths[b]), page)
        n = len(slots)
        if not n:
            continue
        kk = np.stack([k[table[b][j // page], j % page] for j in slots])
        vv = np.stack([v[table[b][j // page], j % page] for j in slots])
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            s = sc * (kk[:, kv] @ q[b, h])
            mag = sc * (np.abs(kk[:, kv]) @ np.abs(q[b, h]))
            ds = ((d + 4) * mag.max() + np.abs(s).max() + np.abs(s - s.max()).max()) * U32
            p = np.exp(s - lse[b, h])
            rel = 2 * ds + 2.0 ** -22 + n * U32
            t_out[b, h] = (rel + n * U32 + 2.0 ** -16) * (p @ np.abs(vv[:, kv]))
            t_lse[b, h] = ds + n * U32 + 2.0 ** -22 + np.abs(lse[b, h]) * U32
            t_mass[b, slots] += rel * p / Hq
    t_mass += (Hq + 2) * U32 * np.abs(mass) + 2.0 ** -126
    return dict(out=out, lse=lse, mass=mass, k=k, v=v, t_out=t_out, t_lse=t_lse, t_mass=t_mass)


def check_attention(x, got, ref, out_dtype):
    half = torch.finfo(out_dtype).eps / 2
    out, lse = bits64(got["out"]), bits64(got["lse"])
    err = np.abs(out - ref["out"])
    bad = ~(err <= ref["t_out"] + half * (np.abs(ref["out"]) + ref["t_out"]) + 2.0 ** -112)
    assert not bad.any(), (int(bad.sum()), float(err[bad].max()))
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(lse), empty)
    e = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, ref["lse"]))
    assert np.all(e <= ref["t_lse"]), float((e - ref["t_lse"]).max())
    if x["mass"] is not None:
        m = bits64(got["mass"])
        e = np.abs(m - ref["mass"])
        assert np.all(e <= ref["t_mass"]), float((e - ref["t_mass"]).max())
        for b, n in enumerate(x["lengths"].tolist()):  # behind a sequence: untouched
            assert np.array_equal(m[b, n:], bits64(x["mass"])[b, n:])


def run_attention(g, **kw):
    """The library's call on GPU tensors; masses go into a copy."""
    from speculative_verification_cover_b200 import dd
    dev = g["q"].device
    B, Hq, d = g["q"].shape
    out = torch.full((B, Hq, d), float("nan"), dtype=g["q"].dtype, device=dev)
    lse = torch.full((B, Hq), float("nan"), device=dev)
    mass_out = None if g["mass"] is None else g["mass"].clone()
    cache = dd.PagedCache(g["k"], g["v"], g["table"])
    dd.dd_paged_attention(g["q"], cache, g["lengths"], out, lse, k_new=g["k_new"], v_new=g["v_new"],
                          mass=g["mass"], mass_out=mass_out, max_len=g["max_len"], **kw)
    return dict(out=out, lse=lse, mass=mass_out)
