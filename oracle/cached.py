"""Token-by-token decoding over a paged cache (oracle, fp64).

Test infrastructure only (see the package docstring). Plain loops over slots and
candidates:

  paged_attention  softmax attention of one token over its cached slots, and the
                   attention mass each slot receives, averaged over the query heads
  evict            the budget rule on (mass, position), and where each slot goes
  beam_select      the K best of all (beam, token) candidates
  fork             page tables and partly filled pages following their parents

The source pages do not cover these; the definitions are the ones in include/dd.h.
"""
from __future__ import annotations

import numpy as np


def held_slots(table_row, length, page_size):
    """Slots of a sequence that lie in a page (a negative page id is a hole)."""
    return [j for j in range(length) if table_row[j // page_size] >= 0]


def paged_attention(q, k_pool, v_pool, table, lengths, k_new=None, v_new=None, mass=None,
                    scale=None):
    """q [B,Hq,d]; pools [P,page,Hkv,d] (changed in place by the append); returns out
    [B,Hq,d], lse [B,Hq] and the masses [B,M] after the step (None without masses: the
    slots a sequence does not have keep what they hold)."""
    B, Hq, d = q.shape
    _, page, Hkv, _ = k_pool.shape
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out = np.zeros((B, Hq, d))
    lse = np.full((B, Hq), -np.inf)
    mass = None if mass is None else np.array(mass, dtype=np.float64)
    for b in range(B):
        n = int(lengths[b])
        slots = held_slots(table[b], n, page)
        if k_new is not None and n > 0:
            if mass is not None:
                mass[b, n - 1] = 0.0
            if n - 1 in slots:
                k_pool[table[b][(n - 1) // page], (n - 1) % page] = k_new[b]
                v_pool[table[b][(n - 1) // page], (n - 1) % page] = v_new[b]
        if not slots:
            continue
        k = np.stack([k_pool[table[b][j // page], j % page] for j in slots])
        v = np.stack([v_pool[table[b][j // page], j % page] for j in slots])
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            s = scale * (k[:, kv] @ q[b, h])
            m = s.max()
            e = np.exp(s - m)
            z = e.sum()
            lse[b, h] = m + np.log(z)
            p = e / z
            out[b, h] = p @ v[:, kv]
            if mass is not None:
                mass[b, slots] += p / Hq
    return out, lse, mass


def evict_one(mass, pos, budget, sink, recent):
    """The old slot of each slot that is left. Kept: protected positions, then the largest
    masses, lower slots first among equals; a kept slot at or beyond the new length fills
    the next freed slot below it."""
    n = len(mass)
    if n <= budget:
        return list(range(n))
    newest = int(max(pos))

    def key(j):
        safe = int(pos[j]) < sink or int(pos[j]) > newest - recent
        weight = -np.inf if np.isnan(mass[j]) else float(mass[j])
        return (0 if safe else 1, 0.0 if safe else -weight, np.isnan(mass[j]) and not safe, j)

    kept = set(sorted(range(n), key=key)[:budget])
    movers = iter(sorted(j for j in kept if j >= budget))
    return [j if j in kept else next(movers) for j in range(budget)]


def beam_candidates(logits, score, done, eos, V, most):
    """(minus score, flat index) of the first `most` candidates of one request, best first;
    equal scores: the lower beam, the larger logit, the lower token."""
    values, places, beams, logit = [], [], [], []
    for k in range(len(score)):
        base = float(score[k])
        if not np.isfinite(base):
            continue
        if done is not None and done[k]:
            values.append(np.array([base]))
            places.append(np.array([k * V + max(eos, 0)]))
            beams.append(np.array([k]))
            logit.append(np.zeros(1))
            continue
        x = np.array(logits[k], dtype=np.float64)
        live = np.isfinite(x)
        if not live.any():
            continue
        m = x[live].max()
        # relative to m: next to logits of 1e30 a log-sum is lost even in 64 bits
        values.append(base + ((x[live] - m) - np.log(np.exp(x[live] - m).sum())))
        places.append(k * V + np.nonzero(live)[0])
        beams.append(np.full(int(live.sum()), k))
        logit.append(x[live])
    if not values:
        return []
    values, places, beams, logit = (np.concatenate(a) for a in (values, places, beams, logit))
    order = np.lexsort((places, -logit, beams, -values))[:most]
    return [(-float(values[i]), int(places[i])) for i in order]


def beam_select(logits, score, done=None, eos=-1):
    """logits [K,V], score [K], done [K]: parent, token, score, done of the K best."""
    K, V = logits.shape
    best = beam_candidates(logits, score, done, eos, V, K)
    parent, token = np.full(K, -1), np.full(K, -1)
    out, ended = np.full(K, -np.inf), np.zeros(K, dtype=np.uint8)
    for r, (neg, at) in enumerate(best):
        k = at // V
        was = done is not None and bool(done[k])
        parent[r], out[r] = k, -neg
        token[r] = eos if was else at % V
        ended[r] = was or token[r] == eos
    return parent, token, out, ended


def parents(parent, K):
    """Row of each beam's parent (an empty slot keeps its own row)."""
    return [n // K * K + (int(p) if 0 <= p < K else n % K) for n, p in enumerate(np.ravel(parent))]


def fork(parent, K, table, lengths, fresh, k_pool, v_pool, table_out):
    """Pools [layers,P,page,Hkv,d] and table_out are changed in place; returns the lengths."""
    page = k_pool.shape[2]
    out = []
    for n, p in enumerate(parents(parent, K)):
        full, rest = divmod(int(lengths[p]), page)
        table_out[n, :full] = table[p, :full]
        if full < table.shape[1]:
            old = int(table[p, full])
            if rest > 0 and old < 0:
                table_out[n, full] = -1
            else:
                table_out[n, full] = fresh[n]
                for pool in (k_pool, v_pool):
                    pool[:, fresh[n], :rest] = pool[:, old, :rest]
        out.append(int(lengths[p]))
    return np.array(out)
