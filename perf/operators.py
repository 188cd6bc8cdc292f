"""Cases of the cached-decoding operators, for timing and for comparing outputs.

Three operators, each in a plain form (elementary torch operations in 32 bits,
64 where scores are ranked) and as the library's calls:

  attention  one new token per sequence over a paged K/V cache, with the token's own
             K/V appended and the attention mass per cached position accumulated
  evict      eviction from that cache by the accumulated mass, down to a budget
  beam       beam search's selection over beams and vocabulary, then the states
             (token history, page tables, the partly filled last pages) reordered:
             full pages are shared, each beam goes on in a fresh page of its own
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _attention(name, B, Hq, Hkv, d, page, min_len, max_len, dtype="bf16", append=True, mass=False,
               holes=False, heads_first=False):
    return {"name": name, "op": "attention", "B": B, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page,
            "min_len": min_len, "max_len": max_len, "dtype": dtype, "append": append, "mass": mass,
            "holes": holes, "heads_first": heads_first}


def _evict(name, B, Hkv, d, page, min_len, max_len, budget, sink, recent, dtype="bf16"):
    return {"name": name, "op": "evict", "B": B, "Hkv": Hkv, "d": d, "page": page, "min_len": min_len,
            "max_len": max_len, "budget": budget, "sink": sink, "recent": recent, "dtype": dtype}


def _beam(name, B, K, V, page, min_len, max_len, layers=1, Hkv=8, d=128, dtype="bf16"):
    return {"name": name, "op": "beam", "B": B, "K": K, "V": V, "page": page, "min_len": min_len,
            "max_len": max_len, "layers": layers, "Hkv": Hkv, "d": d, "dtype": dtype}


def listed():
    return [
        # one user, one layer, a short context: the latency of the call
        _attention("attn_one_short", 1, 32, 8, 128, 16, 200, 200),
        # an interactive server's batch at the contexts of the verification workloads,
        # grouped heads, masses kept for eviction
        _attention("attn_batch16_mass", 16, 32, 8, 128, 16, 333, 1024, mass=True),
        # multi-head (no grouping) over pages stored heads first, odd lengths
        _attention("attn_mha_odd_pages", 7, 32, 32, 128, 48, 101, 2047, heads_first=True),
        # one very long context: everything rides on the split over the length
        _attention("attn_long_one", 1, 32, 8, 128, 64, 131071, 131071),
        # a full server: 64 ragged contexts, seven query heads to a kv head, masses kept
        _attention("attn_batch64_ragged", 64, 28, 4, 128, 32, 17, 8191, mass=True),
        # the exact 32-bit form over pages of 5 tokens, some of them dropped (holes)
        _attention("attn_f32_holes", 5, 10, 2, 64, 5, 1, 1500, dtype="f32", mass=True, holes=True),
        # every step at the budget: one slot leaves each sequence
        _evict("evict_step", 16, 8, 128, 16, 1025, 1025, 1024, 4, 32),
        # long prompts cut down to a budget, once after the prefill
        _evict("evict_prompt", 16, 4, 128, 32, 900, 8192, 1024, 4, 128),
        # a single long cache, odd budget, 32-bit values
        _evict("evict_one_long", 1, 2, 64, 5, 30001, 30001, 9999, 1, 1000, dtype="f32"),
        # one request, four beams, a small vocabulary
        _beam("beam_small", 1, 4, 1000, 16, 70, 70, dtype="f32", Hkv=2, d=64),
        # a batch of requests with the vocabulary of the verification workloads
        _beam("beam_batch8", 8, 8, 126464, 16, 100, 900),
        # many requests, wide beams, the largest vocabulary, two layers' caches
        _beam("beam_batch32_wide", 32, 16, 152064, 32, 33, 500, layers=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "evict", "beam"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    size = 4 if dtype == "f32" else 2
    page = rng.choice([1, 5, 8, 16, 16, 24, 32, 64, 100, 128])
    if op == "attention":
        Hkv = rng.choice([1, 2, 4, 8, 8, 32])
        G = rng.choice([1, 1, 2, 4, 5, 7, 8, 10, 16])
        B = _log(rng, 1, 96)
        most = max(1, min(131072, int(5e8 / (B * Hkv * d * 2 * size))))
        max_len = _log(rng, 1, most)
        return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "d": d, "page": page,
                "min_len": rng.choice([max_len, rng.randint(1, max_len), 1]), "max_len": max_len,
                "dtype": dtype, "append": rng.random() < 0.7, "mass": rng.random() < 0.5,
                "holes": rng.random() < 0.2, "heads_first": rng.random() < 0.3}
    if op == "evict":
        Hkv = rng.choice([1, 2, 4, 8])
        B = _log(rng, 1, 48)
        most = max(40, min(32768, int(2.5e8 / (B * Hkv * d * 2 * size))))
        max_len = _log(rng, 8, most)
        budget = rng.choice([max(1, max_len - 1), rng.randint(1, max_len)])
        sink = min(budget, rng.choice([0, 1, 4]))
        recent = rng.randint(0, (budget - sink) // 2)
        return {"op": op, "B": B, "Hkv": Hkv, "d": d, "page": page,
                "min_len": rng.randint(1, max_len), "max_len": max_len, "budget": budget,
                "sink": sink, "recent": recent, "dtype": dtype}
    K = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 24, 32])
    V = _log(rng, 40, 152064)
    B = _log(rng, 1, max(1, min(64, int(1.5e8 / (K * V * size)))))
    max_len = _log(rng, 1, 600)
    layers = rng.choice([1, 1, 2])
    # no more pages than the widest listed batch has
    B = max(1, min(B, int(4e8 / (K * layers * 8 * d * 2 * size * 3 * page))))
    return {"op": op, "B": B, "K": K, "V": V, "page": page, "min_len": rng.randint(1, max_len),
            "max_len": max_len, "layers": layers, "Hkv": 8, "d": d, "dtype": dtype}


# ------------------------------------------------------------------ inputs
def _lengths(n, lo, hi, gen):
    """n lengths spread evenly over [lo, hi], in an order of the seed's."""
    if n == 1:
        out = torch.tensor([hi])
    else:
        out = lo + (hi - lo) * torch.arange(n) // (n - 1)
    return out[torch.randperm(n, generator=gen)].to(torch.int32)


def _pool(case, pages, layers, gpu):
    """K and V page pools [layers, pages, page, Hkv, d]; heads_first stores a page's
    heads one after the other and gives the same view of it."""
    dt = DTYPES[case["dtype"]]
    P, H, d = case["page"], case["Hkv"], case["d"]
    shape = (layers, pages, H, P, d) if case.get("heads_first") else (layers, pages, P, H, d)
    out = []
    for _ in range(2):
        x = torch.empty(shape, dtype=dt, device="cuda")
        x.normal_(generator=gpu)
        out.append(x.transpose(2, 3) if case.get("heads_first") else x)
    return out


def _tables(counts, width, gen):
    """A page table of `width` columns whose rows own `counts` pages each, in a random
    order of the pool, and the number of pages in use. Unused entries name page 0."""
    n = int(counts.sum())
    ids = torch.randperm(n, generator=gen).to(torch.int32)
    table = torch.zeros(len(counts), width, dtype=torch.int32)
    table[torch.arange(width)[None] < counts[:, None]] = ids
    return table, n


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda").normal_(generator=gpu)
    s = {"case": case}
    if case["op"] == "beam":
        return _prepare_beam(case, s, gen, gpu, normal)
    B, page = case["B"], case["page"]
    dt = DTYPES[case["dtype"]]
    width = -(-case["max_len"] // page)
    lengths = _lengths(B, case["min_len"], case["max_len"], gen)
    if case["op"] == "evict":
        table, n = _tables(torch.full((B,), width), width, gen)
    else:
        table, n = _tables((lengths + page - 1) // page, width, gen)
    k, v = _pool(case, n, 1, gpu)
    s["k"], s["v"] = k[0], v[0]
    if case["op"] == "attention":
        if case["holes"]:
            drop = torch.rand(table.shape, generator=gen) < 0.1
            last = (lengths - 1).clamp(min=0) // page
            drop[torch.arange(B), last.long()] = False
            table[drop] = -1
        s["q"] = (1.5 * normal(B, case["Hq"], case["d"])).to(dt)
        if case["append"]:
            s["k_new"] = normal(B, case["Hkv"], case["d"], dt=dt)
            s["v_new"] = normal(B, case["Hkv"], case["d"], dt=dt)
        s["out"] = torch.zeros(B, case["Hq"], case["d"], dtype=dt, device="cuda")
        s["lse"] = torch.zeros(B, case["Hq"], device="cuda")
        if case["mass"]:
            s["mass"] = normal(B, case["max_len"]).exp_().div_(16)
            s["mass_out"] = torch.zeros(B, case["max_len"], device="cuda")
    else:
        s["mass"] = normal(B, case["max_len"]).mul_(1.5).exp_()
        # slots hold their positions out of order: earlier evictions filled holes with later ones
        pos = torch.zeros(B, case["max_len"], dtype=torch.int32)
        for b, n_b in enumerate(lengths.tolist()):
            pos[b, :n_b] = torch.randperm(n_b, generator=gen).to(torch.int32)
        s["pos"] = pos.cuda()
        s["mass_out"] = torch.zeros_like(s["mass"])
        s["pos_out"] = torch.zeros_like(s["pos"])
        s["lengths_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["table"] = table.cuda()
    s["lengths"] = lengths.cuda()
    return s


def _prepare_beam(case, s, gen, gpu, normal):
    B, K, V, page = case["B"], case["K"], case["V"], case["page"]
    N, dt = B * K, DTYPES[case["dtype"]]
    width = case["max_len"] // page + 1
    per = _lengths(B, case["min_len"], case["max_len"], gen)
    lengths = per.repeat_interleave(K)
    # a request's beams share its full pages; each has a last page of its own, if partly filled
    full, part = per // page, (lengths % page > 0).to(torch.int32)
    shared, n = _tables(full, width, gen)
    table = shared.repeat_interleave(K, 0)
    tails = n + torch.arange(N, dtype=torch.int32)
    rows = torch.arange(N)[part.bool()]
    table[rows, (lengths // page).long()[rows]] = tails[rows]
    s["fresh"] = (n + N + torch.randperm(N, generator=gen).to(torch.int32)).cuda()
    s["k"], s["v"] = _pool(case, n + 2 * N, case["layers"], gpu)
    ld = -(-V // 8) * 8
    logits = normal(B, K, ld, dt=torch.float32).mul_(3.0)
    peak = torch.randint(0, V, (B, K, 1), generator=gpu, device="cuda")
    logits.scatter_add_(2, peak, torch.full((B, K, 1), 8.0, device="cuda"))
    s["logits"] = logits.to(dt)[..., :V]
    score = -normal(B, K).abs().mul_(3.0).add_(20.0)
    s["score"] = score.sort(dim=1, descending=True)[0].contiguous()
    s["eos"] = 2
    s["done"] = (torch.rand(B, K, generator=gpu, device="cuda") < 0.1).to(torch.uint8)
    T = case["max_len"] + 1
    s["history"] = torch.randint(0, V, (B, K, T), generator=gpu, device="cuda", dtype=torch.int32)
    s["table"], s["lengths"] = table.cuda(), lengths.to(torch.int32).cuda()
    for name, like in (("parent", torch.int32), ("token", torch.int32), ("score_out", torch.float32),
                       ("done_out", torch.uint8)):
        s[name] = torch.zeros(B, K, dtype=like, device="cuda")
    s["history_out"] = torch.zeros_like(s["history"])
    s["table_out"] = torch.zeros_like(s["table"])
    s["lengths_out"] = torch.zeros_like(s["lengths"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return RUN[state["case"]["op"]](state)


def _rows(pool, table, page, slots):
    """Pool row (page, offset) of each slot of each sequence; False where the slot's page is a hole."""
    pages = table[torch.arange(table.shape[0], device=table.device)[:, None], slots // page]
    return pages.clamp(min=0).long(), (slots % page).expand(pages.shape), pages >= 0


def _run_attention(s):
    c = s["case"]
    if own:
        from speculative_verification_cover_b200 import dd
        if "cache" not in s:
            s["cache"] = dd.PagedCache(s["k"], s["v"], s["table"])
            s["ws"] = torch.empty(dd.dd_paged_attention_workspace_size(
                c["B"], c["Hq"], c["Hkv"], c["d"], c["max_len"], c["mass"]), dtype=torch.uint8,
                device="cuda")
        dd.dd_paged_attention(s["q"], s["cache"], s["lengths"], s["out"], s["lse"],
                              k_new=s.get("k_new"), v_new=s.get("v_new"), mass=s.get("mass"),
                              mass_out=s.get("mass_out"), max_len=c["max_len"], workspace=s["ws"])
    else:
        B, Hq, Hkv, page, n = c["B"], c["Hq"], c["Hkv"], c["page"], c["max_len"]
        lengths = s["lengths"].long()
        if c["append"]:
            last = (lengths - 1)[:, None]
            p, o, ok = _rows(s["k"], s["table"], page, last)
            s["k"][p[:, 0], o[:, 0]] = s["k_new"]
            s["v"][p[:, 0], o[:, 0]] = s["v_new"]
        slots = torch.arange(n, device="cuda")[None]
        p, o, ok = _rows(s["k"], s["table"], page, slots)
        ok = ok & (slots < lengths[:, None])
        k = s["k"][p, o].float()
        q = s["q"].float().view(B, Hkv, Hq // Hkv, -1)
        x = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(c["d"])
        del k
        x = torch.where(ok[:, None, None], x, -math.inf)
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
        z = e.sum(-1, keepdim=True)
        prob = e / torch.where(z > 0, z, 1.0)
        v = torch.where(ok[..., None, None], s["v"][p, o].float(), 0.0)
        s["out"].copy_(torch.matmul(prob, v.permute(0, 2, 1, 3)).view(B, Hq, -1))
        s["lse"].copy_((m + torch.log(z)).view(B, Hq))
        if c["mass"]:
            before = s["mass"]
            if c["append"]:
                before = torch.where(slots == (lengths - 1)[:, None], 0.0, before)
            after = before + prob.sum((1, 2)) / Hq
            s["mass_out"].copy_(torch.where(slots < lengths[:, None], after, s["mass_out"]))
    got = {"out": s["out"], "lse": s["lse"]}
    if c["mass"]:
        got["mass"] = s["mass_out"]
    if c["append"]:
        got["k"], got["v"] = s["k"], s["v"]
    return got


def _run_evict(s):
    c = s["case"]
    if own:
        from speculative_verification_cover_b200 import dd
        if "cache" not in s:
            s["cache"] = dd.PagedCache(s["k"], s["v"], s["table"])
        dd.dd_cache_evict(s["cache"], s["lengths"], s["mass"], s["pos"], c["budget"], s["mass_out"],
                          s["pos_out"], s["lengths_out"], sink=c["sink"], recent=c["recent"])
    else:
        n, budget, page = c["max_len"], min(c["budget"], c["max_len"]), c["page"]
        slots = torch.arange(n, device="cuda")[None]
        lengths = s["lengths"].long()[:, None]
        used = slots < lengths
        pos = torch.where(used, s["pos"], -1)
        top = pos.amax(1, keepdim=True)
        keep_first = used & ((pos < c["sink"]) | (pos > top - c["recent"]))
        key = torch.where(keep_first, math.inf, torch.where(used, s["mass"], -math.inf))
        order = torch.argsort(key, dim=1, descending=True, stable=True)
        kept = torch.zeros_like(used).scatter_(1, order[:, :budget], True) & used
        after = lengths.clamp(max=budget)
        hole = ~kept & (slots < after)
        source = torch.where(kept & (slots >= after), slots, n).sort(dim=1)[0]
        rank = (hole.long().cumsum(1) - 1).clamp(min=0)
        src = torch.where(hole, source.gather(1, rank).clamp(max=n - 1), slots.expand_as(hole))
        to = slots[:, :budget]
        p0, o0, _ = _rows(s["k"], s["table"], page, src[:, :budget])
        p1, o1, _ = _rows(s["k"], s["table"], page, to)
        for x in (s["k"], s["v"]):
            x[p1, o1] = x[p0, o0]
        left = slots < after
        s["mass_out"].copy_(torch.where(left, s["mass"].gather(1, src), s["mass_out"]))
        s["pos_out"].copy_(torch.where(left, s["pos"].gather(1, src), s["pos_out"]))
        s["lengths_out"].copy_(after[:, 0])
    return {"lengths": s["lengths_out"], "mass": s["mass_out"], "pos": s["pos_out"], "k": s["k"],
            "v": s["v"]}


def _run_beam(s):
    c = s["case"]
    B, K, V, page = c["B"], c["K"], c["V"], c["page"]
    if own:
        from speculative_verification_cover_b200 import dd
        if "cache" not in s:
            s["cache"] = dd.PagedCache(s["k"], s["v"], s["table"])
            s["ws"] = torch.empty(dd.dd_beam_select_workspace_size(B, K, V, s["logits"].dtype),
                                  dtype=torch.uint8, device="cuda")
        dd.dd_beam_select(s["logits"], s["score"], s["parent"], s["token"], s["score_out"],
                          done=s["done"], done_out=s["done_out"], eos=s["eos"], workspace=s["ws"])
        dd.dd_beam_reorder(s["parent"], [(s["history"], s["history_out"])])
        dd.dd_paged_fork(s["cache"], s["parent"], s["lengths"], s["fresh"], s["table_out"],
                         s["lengths_out"])
    else:
        x = s["logits"].double()
        m = x.amax(-1, keepdim=True)
        lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
        at = torch.arange(V, device="cuda")
        done = s["done"].bool()[..., None]
        ended = torch.where(at == s["eos"], 0.0, -math.inf)
        total = s["score"].double()[..., None] + torch.where(done, ended, x - lse)
        flat = total.view(B, K * V)
        best, cand = torch.sort(flat, dim=1, descending=True, stable=True)
        best, cand = best[:, :K], cand[:, :K]
        s["parent"].copy_(cand // V)
        s["token"].copy_(cand % V)
        s["score_out"].copy_(best)
        parent = s["parent"].long()
        s["done_out"].copy_(s["done"].gather(1, parent) | (s["token"] == s["eos"]).to(torch.uint8))
        row = (torch.arange(B, device="cuda")[:, None] * K + parent).view(-1)
        s["history_out"].copy_(s["history"].view(B * K, -1)[row].view(s["history"].shape))
        lengths = s["lengths"][row].long()
        full, rest = lengths // page, lengths % page
        table = s["table"][row]
        cols = torch.arange(table.shape[1], device="cuda")[None]
        old = table.gather(1, full[:, None].clamp(max=table.shape[1] - 1))[:, 0].long()
        new = torch.where(cols == full[:, None], s["fresh"][:, None], table)
        used = cols <= full[:, None]
        s["table_out"].copy_(torch.where(used, new, s["table_out"]))
        s["lengths_out"].copy_(lengths)
        fresh = s["fresh"].long()
        take = (torch.arange(page, device="cuda")[None] < rest[:, None])[None, :, :, None, None]
        for x in (s["k"], s["v"]):
            x[:, fresh] = torch.where(take, x[:, old], x[:, fresh])
    return {"parent": s["parent"], "token": s["token"], "score": s["score_out"], "done": s["done_out"],
            "history": s["history_out"], "table": s["table_out"], "lengths": s["lengths_out"],
            "k": s["k"], "v": s["v"]}


RUN = {"attention": _run_attention, "evict": _run_evict, "beam": _run_beam}


# ------------------------------------------------------------------ what a pass cannot do without
def _total(case):
    n = case["B"]
    if n == 1:
        return case["max_len"]
    lo, hi = case["min_len"], case["max_len"]
    return sum(lo + (hi - lo) * i // (n - 1) for i in range(n))


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    B, d, Hkv, tokens = case["B"], case["d"], case["Hkv"], _total(case)
    row = 2 * Hkv * d * size  # a token's K and V
    if case["op"] == "attention":
        held = 0.9 if case["holes"] else 1.0
        new = 2 * row * B if case["append"] else 0  # read once, written to the cache once
        return {"bytes": held * tokens * row + new + 2 * B * case["Hq"] * d * size + 4 * B * case["Hq"]
                + 4 * B + 4 * -(-tokens // case["page"]) + (8 * tokens if case["mass"] else 0),
                "flops": 4.0 * held * tokens * case["Hq"] * d}
    if case["op"] == "evict":
        lo, hi = case["min_len"], case["max_len"]
        each = [lo + (hi - lo) * i // max(1, B - 1) if B > 1 else hi for i in range(B)]
        left = [min(n, case["budget"]) for n in each]
        # a slot is kept with chance budget / length, so this share of the kept lie behind the budget
        moved = sum(l * (1.0 - l / n) for l, n in zip(left, each))
        return {"bytes": 8.0 * tokens + 8.0 * sum(left) + 2 * row * moved + 8 * B, "flops": float(tokens)}
    K, V, page = case["K"], case["V"], case["page"]
    lo, hi = case["min_len"], case["max_len"]
    each = [lo + (hi - lo) * i // max(1, B - 1) if B > 1 else hi for i in range(B)]
    partial = sum(n % page for n in each) * K
    entries = sum(n // page + 1 for n in each) * K
    return {"bytes": B * K * V * size + 26.0 * B * K + 8.0 * B * K * (case["max_len"] + 1) + 8.0 * entries
            + 8.0 * B * K + 2.0 * row * case["layers"] * partial, "flops": 4.0 * B * K * V}


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    return EXACT[case["op"]](case, prepare(case, seed))


def _exact_attention(c, s):
    B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    mass = s["mass_out"].double() if c["mass"] else None
    for b, n in enumerate(s["lengths"].tolist()):
        entries = s["table"][b, : -(-n // page)].tolist()
        held = torch.tensor([j for j in range(n) if entries[j // page] >= 0], device="cuda")
        ids = s["table"][b].long()[held // page]
        k, v = s["k"][ids, held % page].double(), s["v"][ids, held % page].double()
        if c["append"] and len(held) and int(held[-1]) == n - 1:
            k[-1], v[-1] = s["k_new"][b].double(), s["v_new"][b].double()
        if mass is not None:
            mass[b, :n] = s["mass"][b, :n].double()
            if c["append"]:
                mass[b, n - 1] = 0.0
        for h in range(Hkv):
            logit = k[:, h] @ s["q"][b, h * G:(h + 1) * G].double().T / d ** 0.5  # [held, G]
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(logit, 0)
            weight = torch.softmax(logit, 0)
            out[b, h * G:(h + 1) * G] = weight.T @ v[:, h]
            if mass is not None:
                mass[b].index_add_(0, held, weight.sum(1) / Hq)
    got = {"out": out, "lse": lse}
    if c["mass"]:
        got["mass"] = mass
    if c["append"]:
        got["k"] = got["v"] = None  # copies of the inputs
    return got


def _exact_evict(c, s):
    lengths = s["lengths_out"].clone()
    mass, pos = s["mass_out"].double(), s["pos_out"].clone()
    masses, positions = s["mass"].double().cpu().tolist(), s["pos"].cpu().tolist()
    k, v, table = s["k"], s["v"], s["table"].cpu().tolist()
    for b, n in enumerate(s["lengths"].tolist()):
        newest = max(positions[b][:n])
        bound = lambda j: positions[b][j] < c["sink"] or positions[b][j] > newest - c["recent"]
        ranked = sorted(range(n), key=lambda j: (not bound(j), -masses[b][j], j))
        kept = set(ranked[: c["budget"]])
        left = len(kept)
        holes = [j for j in range(left) if j not in kept]
        movers = sorted(j for j in kept if j >= left)
        src = list(range(left))
        for h, j in zip(holes, movers):
            src[h] = j
        where = lambda js: (torch.tensor([table[b][j // c["page"]] for j in js], device="cuda"),
                            torch.tensor([j % c["page"] for j in js], device="cuda"))
        if holes:
            (p1, o1), (p0, o0) = where(holes), where(movers)
            k[p1, o1] = k[p0, o0]
            v[p1, o1] = v[p0, o0]
        lengths[b] = left
        mass[b, :left] = torch.tensor([masses[b][j] for j in src], device="cuda", dtype=torch.float64)
        pos[b, :left] = torch.tensor([positions[b][j] for j in src], device="cuda", dtype=torch.int32)
    return {"lengths": lengths, "mass": mass, "pos": pos, "k": k.double(), "v": v.double()}


def _exact_beam(c, s):
    B, K, V, page = c["B"], c["K"], c["V"], c["page"]
    score = torch.zeros(B, K, dtype=torch.float64, device="cuda")
    parent, token, done = torch.zeros_like(s["parent"]), torch.zeros_like(s["token"]), torch.zeros_like(s["done"])
    for b in range(B):
        found = []
        for k in range(K):
            base = float(s["score"][b, k])
            if s["done"][b, k]:
                found.append((-base, k * V + s["eos"]))
                continue
            x = s["logits"][b, k].double()
            logp = (x - torch.logsumexp(x, 0)).cpu().numpy()
            top = (-logp).argsort(kind="stable")[:K]
            found += [(-(base + float(logp[i])), k * V + int(i)) for i in top]
        for r, (neg, at) in enumerate(sorted(found)[:K]):
            score[b, r], parent[b, r], token[b, r] = -neg, at // V, at % V
            done[b, r] = int(bool(s["done"][b, at // V]) or at % V == s["eos"])
    history, table, lengths = s["history_out"].clone(), s["table_out"].clone(), s["lengths_out"].clone()
    old_table, old_len, fresh = s["table"].tolist(), s["lengths"].tolist(), s["fresh"].tolist()
    kv = (s["k"], s["v"])
    came = parent.tolist()
    for n in range(B * K):
        p = n // K * K + came[n // K][n % K]
        history.view(B * K, -1)[n] = s["history"].view(B * K, -1)[p]
        length = old_len[p]
        lengths[n] = length
        row = old_table[p][: length // page]
        if length % page:
            last = old_table[p][length // page]
            for x in kv:
                x[:, fresh[n], : length % page] = x[:, last, : length % page]
        row.append(fresh[n])
        table[n, : len(row)] = torch.tensor(row, dtype=torch.int32, device="cuda")
    return {"parent": parent, "token": token, "score": score, "done": done, "history": history,
            "table": table, "lengths": lengths, "k": kv[0].double(), "v": kv[1].double()}


EXACT = {"attention": _exact_attention, "evict": _exact_evict, "beam": _exact_beam}
