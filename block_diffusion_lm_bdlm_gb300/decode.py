"""Block-by-block answering over a paged 8-bit cache: the order of the
bdlm_cache_* calls that one model's attention layers need.

    dec = BlockDecoder(cache, block=32)
    cu = dec.begin(rows)              # rows: int32 [n_seqs], new rows of every sequence (0: takes no part)
    for step in range(steps):         # a prompt takes one step, a block several: its rows are written anew in each
        for layer in range(n_layers):
            o, _ = dec.attend(layer, q, k, v)
    ...                               # keep the rows: begin the next block; or dec.rewind() and begin again
    dec.branch(parents, children)     # candidates that share what was written so far; behind a block's last step
    dec.end(seqs)                     # their pages are free again

All state is on the device, the cache's table and lens and the present block's
offsets: begin, attend, rewind, branch and end only launch work on the current
stream and can be captured into graphs. begin's first step of a whole prompt
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

from . import PageCache, bdlm_cache_attn_fwd, bdlm_cache_fork, bdlm_cache_reserve, bdlm_cache_write


_NONE = -2 ** 31


class BlockDecoder:
    def __init__(self, cache: PageCache, block: int, softmax_scale: float = 0.0):
        if block < 1:
            raise ValueError("block must be positive")
        self.cache, self.block, self.softmax_scale = cache, int(block), float(softmax_scale)
        self.cu_rows = torch.zeros(cache.n_seqs + 1, dtype=torch.int32, device=cache.device)
        self._cu = torch.zeros_like(self.cu_rows)  # those of cu_rows that attend goes by: all 0 once the block is over
        self._kept = cache.lens.clone()            # lengths before the last begin
        self._rows = torch.zeros_like(cache.lens)  # rows that it gave and rewind may still take; _NONE: none

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
        return self.cu_rows

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
        return bdlm_cache_attn_fwd(self.cache, q, self._cu, self.block, layer=layer, q_pos=self._kept,
                                   softmax_scale=self.softmax_scale, out=out, lse=lse, check=check)

    def rewind(self) -> None:
        """Drop the rows of the last begin. Sequences that have ended or
        branched off since then stay as they are."""
        lens = self.cache.lens
        lens.copy_(torch.where(self._untouched(), self._kept, lens))
        self._cu.zero_()

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

    def end(self, seqs: torch.Tensor) -> None:
        """Empty the sequences; pages that no other one names are free. seqs
        holds their numbers (int32 or int64; negative ones count from the end);
        a number that no sequence has is passed over."""
        self.cache.lens.masked_fill_(self._named(seqs), 0)
        self._settle()

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
