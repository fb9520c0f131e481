"""Block-by-block answering over a paged 8-bit cache: the order of the
bdlm_cache_* calls that one model's attention layers need.

    dec = BlockDecoder(cache, block=32)
    cu = dec.begin(rows)              # rows: int32 [n_seqs], new rows of every sequence (0: takes no part)
    for step in range(steps):         # a prompt takes one step, a block several: its rows are written anew in each
        for layer in range(n_layers):
            o, _ = dec.attend(layer, q, k, v)
        left = dec.choose(tokens, logits, u, mask_id)  # draw tokens, keep the surest; rows still masked
    ...                               # keep the rows: begin the next block; or dec.rewind() and begin again
    dec.branch(parents, children)     # candidates that share what was written so far; behind a block's last step
    dec.end(seqs)                     # their pages are free again

With share=True the candidates' attention reads the pages that they share once
for all of them: begin finds the runs of neighbouring sequences that do
(bdlm_cache_prefixes), so children should be numbered side by side.

All state is on the device, the cache's table and lens and the present block's
offsets: begin, attend, choose, rewind, branch and end only launch work on the
current stream and can be captured into graphs. begin's first step of a whole prompt
and a denoising step of one block are the same call: under the block-causal
mask a prompt's rows see the blocks up to their own, and the rows of a block
that starts at a block boundary see everything before it and each other.

A page has one scale for each head, so a step rounds the committed rows of a
page that its own rows share anew whenever it changes that scale: values below
2^-6 of a larger scale lose bits, or become 0, and a later step with smaller
rows does not bring them back. Where that matters, let every block (and the
prompt's end) lie on a page boundary: with pages that divide the block, and
prompts filled up to whole pages, a step's pages hold its own rows only.
"""
from __future__ import annotations

import torch

from . import (PageCache, bdlm_cache_attn_fwd, bdlm_cache_attn_shared_fwd, bdlm_cache_fork, bdlm_cache_prefixes,
               bdlm_cache_reserve, bdlm_cache_write, bdlm_sample, bdlm_unmask)


_NONE = -2 ** 31


class BlockDecoder:
    def __init__(self, cache: PageCache, block: int, softmax_scale: float = 0.0, share: bool = False):
        if block < 1:
            raise ValueError("block must be positive")
        self.cache, self.block, self.softmax_scale = cache, int(block), float(softmax_scale)
        self.cu_rows = torch.zeros(cache.n_seqs + 1, dtype=torch.int32, device=cache.device)
        self._cu = torch.zeros_like(self.cu_rows)  # those of cu_rows that attend goes by: all 0 once the block is over
        self._kept = cache.lens.clone()            # lengths before the last begin
        self._rows = torch.zeros_like(cache.lens)  # rows that it gave and rewind may still take; _NONE: none
        self._runs = torch.empty((3, cache.n_seqs), dtype=torch.int32, device=cache.device) if share else None
        self._plan()

    def begin(self, rows: torch.Tensor, *, check: bool = False) -> torch.Tensor:
        """Make room for `rows` new rows of every sequence behind what it
        holds; returns their offsets (int32 [n_seqs + 1]). If the cache has no
        room, rows are negative, or a sequence would grow inside a page that
        another one reads too (one that was rewound behind a branch), no
        sequence gets any row: the offsets are all 0, so that attend does
        nothing, and check=True raises."""
        want = self.cache.lens + rows
        want.masked_fill_(want < self.cache.lens, -1)  # too many rows, or fewer than none: refused like no room
        self._kept.copy_(self.cache.lens)
        try:
            bdlm_cache_reserve(self.cache, want, check=check)
        finally:  # also where that raises: the rows of the block before are no longer to be written
            torch.sub(self.cache.lens, self._kept, out=self._rows)
            torch.cumsum(self._rows, 0, dtype=torch.int32, out=self._cu[1:])
            self.cu_rows.copy_(self._cu)
            self._plan()
        return self.cu_rows

    def _plan(self) -> None:
        """Which sequences' rows read which pages together, from here on."""
        if self._runs is not None:
            bdlm_cache_prefixes(self.cache, self._cu, q_pos=self._kept, out=self._runs)

    def attend(self, layer: int, q, k, v, *, out=None, lse=None, check: bool = False):
        """Write the rows' keys and values and attend; (o, lse). The rows of a
        sequence that has ended since begin are not written and see nothing
        (o = 0, lse = -inf); the others keep their places in q, k and v. After
        rewind there are no rows until the next begin, and o and lse stay
        unwritten. check=True synchronises and raises where no sequence has
        rows or the offsets do not fit q."""
        if check and q.shape[0] > 0 and int(self._cu[-1]) == 0:
            raise RuntimeError("no sequence has rows: begin a block before attend")
        bdlm_cache_write(self.cache, k, v, self._cu, layer=layer)
        # The positions come from begin: lengths say nothing about those of a sequence that has ended.
        more = dict(layer=layer, q_pos=self._kept, softmax_scale=self.softmax_scale, out=out, lse=lse, check=check)
        if self._runs is None:
            return bdlm_cache_attn_fwd(self.cache, q, self._cu, self.block, **more)
        return bdlm_cache_attn_shared_fwd(self.cache, q, self._cu, self.block, self._runs, **more)

    def choose(self, tokens, logits, u, mask_id: int, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, n_min=1,
               threshold=float("nan"), check: bool = False) -> torch.Tensor:
        """Draw a token for every row that has none yet (tokens[i] == mask_id;
        int32, a row of logits and of u for each) and enter, in tokens, those
        with a log-probability of at least `threshold` (NaN: none) and at
        least the n_min surest of every sequence. mask_id itself is never
        drawn: where it is a token of the vocabulary its logit counts as -inf,
        for the log-probabilities as well. Returns the rows of each sequence
        that are still masked (int32 [n_seqs])."""
        drawn, logprob = torch.empty_like(tokens), torch.empty_like(u)
        bdlm_sample(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, tokens=tokens,
                    mask_id=mask_id, out=drawn, logprob=logprob, draw_mask=False)
        return bdlm_unmask(tokens, drawn, logprob, self._cu, mask_id, n_min=n_min, threshold=threshold, out=tokens,
                           check=check)[1]

    def rewind(self) -> None:
        """Drop the rows of the last begin. Sequences that have ended or
        branched off since then stay as they are."""
        lens = self.cache.lens
        lens.copy_(torch.where(self._untouched(), self._kept, lens))
        self._cu.zero_()
        self._plan()

    def _untouched(self) -> torch.Tensor:
        """The sequences whose lengths are those that begin left."""
        return self.cache.lens - self._kept == self._rows

    def _settle(self) -> None:
        """Take the others out of rewind's reach, before their lengths can
        come to those of begin again."""
        self._rows.masked_fill_(~self._untouched(), _NONE)

    def branch(self, parents: torch.Tensor, children: torch.Tensor, *, check: bool = False) -> None:
        """children[i] (empty) continue what parents[i] hold. Where that shares
        a page with rows of the present block, or a child has rows in it, the
        block is over: as after rewind there are no rows until the next begin,
        since another step would write into what the candidates share."""
        self._settle()
        before = self.cache.lens.clone()
        bdlm_cache_fork(self.cache, parents, children, check=check)
        lens, page = self.cache.lens, self.cache.page
        took = self._cu[1:] > self._cu[:-1]
        shared = took & (lens // page * page > self._kept) & self._named(parents)  # below lens // page * page pages are shared
        over = (shared | took & self._named(children)).any() & (lens != before).any()  # a fork that failed shares nothing
        self._cu.masked_fill_(over, 0)
        self._plan()

    def end(self, seqs: torch.Tensor) -> None:
        """Empty the sequences; pages that no other one names are free. seqs
        holds their numbers (int32 or int64; negative ones count from the end);
        a number that no sequence has is passed over."""
        self.cache.lens.masked_fill_(self._named(seqs), 0)
        self._settle()
        self._plan()

    def _named(self, seqs: torch.Tensor) -> torch.Tensor:
        """Which sequences the numbers name (bool [n_seqs]). A number out of
        range must not index anything: on the device that ends the process."""
        if seqs.dtype not in (torch.int32, torch.int64):
            raise ValueError(f"sequence numbers must be int32 or int64, got {seqs.dtype}")
        n = self.cache.n_seqs
        at = seqs.to(self.cache.device, torch.int64).reshape(-1)
        at = torch.where(at < 0, at + n, at)
        hit = torch.zeros(n + 1, dtype=torch.bool, device=self.cache.device)
        return hit.index_fill_(0, torch.where((at < 0) | (at >= n), n, at), True)[:n]
