"""Token-by-token decoding on the cached operators, composed as a program uses them.

BudgetedCache  one layer's cache of N sequences held at a slot budget: attention of each
               new token (appending it, adding up the masses), eviction by those masses.
BeamDecode     beam search over the layers of a model: each beam's caches share the pages
               their histories share; a step attends in every layer, selects over beams
               and vocabulary, and moves every state to its new beam.

Both hold their buffers from the start and stay on the device; the model around them (its
projections and logits) is the caller's. Prompts come in the layout of the verification
step's attention, [N,L,Hkv,d], and its d_in can serve as the first masses.
"""
from __future__ import annotations

import torch

from . import dd


def _pages(slots, page_size):
    return -(-slots // page_size)


class BudgetedCache:
    def __init__(self, N, Hq, Hkv, d, budget, page_size=16, sink=4, recent=32, every=1,
                 prompt=0, dtype=torch.bfloat16, device="cuda"):
        """budget: slots a sequence keeps; every: tokens between evictions (the cache has room
        for budget + every slots); prompt: the longest prompt, if it is above the budget."""
        if budget < 1 or every < 1 or prompt < 0:
            raise ValueError(f"budget {budget} and every {every} must be positive, prompt {prompt} not negative")
        if sink < 0 or recent < 0 or sink + recent > budget:
            raise ValueError(f"sink {sink} and recent {recent} must fit into the budget of {budget} slots")
        cap = max(budget + every, prompt)
        width = _pages(cap, page_size)
        self.N, self.Hq, self.budget, self.every = N, Hq, budget, every
        self.sink, self.recent = sink, recent
        shape = (N * width, page_size, Hkv, d)
        table = torch.arange(N * width, dtype=torch.int32, device=device).view(N, width)
        self.cache = dd.PagedCache(torch.zeros(shape, dtype=dtype, device=device),
                                   torch.zeros(shape, dtype=dtype, device=device), table)
        cap = self.cache.slots
        self.lengths = torch.zeros(N, dtype=torch.int32, device=device)
        self.seen = torch.zeros(N, dtype=torch.int32, device=device)  # positions so far
        self.mass = torch.zeros(N, cap, device=device)
        self.pos = torch.zeros(N, cap, dtype=torch.int32, device=device)
        # what an eviction writes; it and the buffers above change places
        self._other = (torch.zeros_like(self.lengths), torch.zeros_like(self.mass),
                       torch.zeros_like(self.pos))
        self.out = torch.empty(N, Hq, d, dtype=dtype, device=device)
        self.lse = torch.empty(N, Hq, device=device)
        self.ws = torch.empty(dd.dd_paged_attention_workspace_size(N, Hq, Hkv, d, cap, True),
                              dtype=torch.uint8, device=device)
        self._most = 0  # no sequence holds more slots than this

    def fill(self, k, v, mass=None, lengths=None):
        """A prompt: k, v [N,L,Hkv,d]; mass [N,L] its first masses (dd_dualview_attention's
        d_in, say; None: zero); lengths [N] its lengths (None: L; values outside 0 .. L are
        clamped)."""
        N, L = k.shape[:2]
        if L > self.cache.slots:
            raise ValueError(f"a prompt of {L} slots, room for {self.cache.slots}")
        page = self.cache.page_size
        slots = torch.arange(L, device=k.device)
        pages, rows = self.cache.page_table[:, slots // page].long(), slots % page
        self.cache.k[pages, rows] = k
        self.cache.v[pages, rows] = v
        self.mass.zero_()
        if mass is not None:
            self.mass[:, :L] = mass
        self.pos[:, :L] = slots.to(torch.int32)
        # what attend() makes slot indexes of: no length may lie behind the rows
        self.lengths.fill_(L) if lengths is None else self.lengths.copy_(lengths.clamp(0, L))
        self.seen.copy_(self.lengths)
        self._most = L
        if L > self.budget:
            self.evict()

    def attend(self, q, k_new, v_new):
        """One token per sequence: out [N,Hq,d] (the same buffer every time)."""
        if self._most >= self.budget + self.every:
            self.evict()
        self.lengths += 1
        self.pos.scatter_(1, (self.lengths - 1).long()[:, None], self.seen[:, None])
        self.seen += 1
        self._most += 1
        dd.dd_paged_attention(q, self.cache, self.lengths, self.out, self.lse, k_new=k_new,
                              v_new=v_new, mass=self.mass, mass_out=self.mass, workspace=self.ws)
        return self.out

    def evict(self):
        lengths, mass, pos = self._other
        dd.dd_cache_evict(self.cache, self.lengths, self.mass, self.pos, self.budget, mass, pos,
                          lengths, sink=self.sink, recent=self.recent)
        self._other = (self.lengths, self.mass, self.pos)
        self.lengths, self.mass, self.pos = lengths, mass, pos
        self._most = min(self._most, self.budget)


class BeamDecode:
    def __init__(self, k, v, Hq, K, vocab, steps, page_size=16, eos=-1):
        """k, v [layers,B,L,Hkv,d]: the prompts' caches, one beam each; K beams and at most
        `steps` tokens (begin) and `steps` choices (advance) from there on, in any order: the
        first choice may come from the prompts' own logits, before any token."""
        layers, B, L, Hkv, d = k.shape
        dev, dtype, N = k.device, k.dtype, B * K
        i32 = dict(dtype=torch.int32, device=dev)
        self.B, self.K, self.N, self.L, self.eos, self.steps = B, K, N, L, eos, steps
        shared = L // page_size                    # full prompt pages, one set per request
        width = (L + steps) // page_size + 1
        # Pages a beam may write: two for every page it can reach. A fork copies a beam's
        # open page out of one of them and into the other; the one it left is read by no
        # beam any more when the next fork writes it.
        self._first = B * shared
        self._own = torch.arange(N, **i32)
        pages = self._first + 2 * N * (width - shared)
        shape = (layers, pages, page_size, Hkv, d)
        self.pool_k, self.pool_v = (torch.zeros(shape, dtype=dtype, device=dev) for _ in range(2))
        self.table = torch.zeros(N, width, **i32)
        self._table_out = torch.zeros_like(self.table)
        self.caches = [dd.PagedCache(self.pool_k, self.pool_v, t) for t in (self.table, self._table_out)]
        self._layers = [[c.layer(i) for i in range(layers)] for c in self.caches]
        self.lengths = torch.full((N,), L, **i32)
        self._lengths_out = torch.zeros_like(self.lengths)
        self.score = torch.full((B, K), float("-inf"), device=dev)
        self.score[:, 0] = 0.0                     # the other beams come out of the first
        self._score_out = torch.zeros_like(self.score)
        self.done = torch.zeros(B, K, dtype=torch.uint8, device=dev)
        self._done_out = torch.zeros_like(self.done)
        self.tokens = torch.zeros(B, K, steps, **i32)
        self._tokens_out = torch.zeros_like(self.tokens)
        self.parent, self.token = torch.zeros(B, K, **i32), torch.zeros(B, K, **i32)
        self.out = torch.empty(N, Hq, d, dtype=dtype, device=dev)
        self.ws = torch.empty(max(
            dd.dd_paged_attention_workspace_size(N, Hq, Hkv, d, width * page_size),
            dd.dd_beam_select_workspace_size(B, K, vocab, torch.float32)), dtype=torch.uint8, device=dev)
        self.t = 0        # choices so far
        self._slots = L   # a beam's slots
        # the prompts: full pages shared by a request's beams, the rest in each beam's own page
        page = page_size
        if shared:
            for pool, x in ((self.pool_k, k), (self.pool_v, v)):
                pool[:, :self._first] = x[:, :, :shared * page].reshape(layers, B * shared, page, Hkv, d)
            ids = torch.arange(B * shared, **i32).view(B, shared)
            self.table[:, :shared] = ids.repeat_interleave(K, 0)
        own = self._fresh()
        self.table[:, shared] = own
        self._open = shared  # the last page a beam has
        rest = L - shared * page
        for pool, x in ((self.pool_k, k), (self.pool_v, v)):
            pool[:, own.long(), :rest] = x[:, :, shared * page:].repeat_interleave(K, 1)

    def _fresh(self):
        """The page each beam goes on in: one of the two of the page its next slot lies in."""
        page = self.caches[0].page_size
        i = self._slots // page - self.L // page
        return self._first + 2 * (i * self.N + self._own) + self.t % 2

    def begin(self):
        """A new token for every beam: its slot counts from here on."""
        if self._slots - self.L >= self.steps:
            raise ValueError(f"all {self.steps} steps are taken")
        page = self._slots // self.caches[0].page_size
        if page > self._open:  # the last token filled a page, and no fork gave a next one
            self.table[:, page] = self._fresh()
            self._open = page
        self.lengths += 1
        self._slots += 1

    def attend(self, layer, q, k_new, v_new):
        """One layer: q [N,Hq,d], k_new, v_new [N,Hkv,d] of the beams' current tokens."""
        dd.dd_paged_attention(q, self._layers[0][layer], self.lengths, self.out, k_new=k_new,
                              v_new=v_new, workspace=self.ws)
        return self.out

    def advance(self, logits):
        """logits [B,K,V] of the beams: selects, and moves every state to its new beam. The
        chosen tokens [B,K] are what the beams' next step embeds (-1: no candidate was left for
        that beam, its score is -inf)."""
        if self.t >= self.steps:
            raise ValueError(f"all {self.steps} steps are taken")
        dd.dd_beam_select(logits, self.score, self.parent, self.token, self._score_out,
                          done=self.done, done_out=self._done_out, eos=self.eos, workspace=self.ws)
        dd.dd_beam_reorder(self.parent, [(self.tokens, self._tokens_out)])
        self.tokens, self._tokens_out = self._tokens_out, self.tokens
        self.tokens[:, :, self.t] = self.token
        self.t += 1
        dd.dd_paged_fork(self.caches[0], self.parent, self.lengths, self._fresh(), self._table_out,
                         self._lengths_out)
        self._open = self._slots // self.caches[0].page_size
        self.table, self._table_out = self._table_out, self.table
        self.caches.reverse()
        self._layers.reverse()
        self.lengths, self._lengths_out = self._lengths_out, self.lengths
        self.score, self._score_out = self._score_out, self.score
        self.done, self._done_out = self._done_out, self.done
        return self.token
