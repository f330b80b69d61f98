"""Beam search of a one-layer toy target over a paged cache, every step on the device.

A step of a batch of requests with some beams each:

  tokens  -> forward                      kv_append and paged_attention over every beam's pages
  logits  -> sv.beam_select               the best continuations over beams and vocabulary
  state   -> sv.beam_reorder              histories and marks follow their parents, in place
  pages   -> sv.kv_fork                   beams share what they have in common, and get room for a token
          -> sv.kv_copy                   begun pages that several beams would write on

A finished beam gives its pages back and stays among the beams with its score.  So does one that the pool has no pages
for, and the beams of a request whose logits are NaN: their text ends there, and nothing is appended to them.  Weights
are random, so the text means nothing.  Run: python examples/beam_search.py [--requests 16] [--beams 4] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from speculative_decoding_verification_rows_gb300 import sv  # noqa: E402
from target_step import Target  # noqa: E402


class BeamSearch:
    """`beams` beams for each of n requests; request i's are rows i * beams .. of the page table."""

    def __init__(self, target: Target, n: int, beams: int, steps: int, end_token: int):
        device, rows = target.device, n * beams
        self.t, self.n, self.beams, self.end = target, n, beams, end_token
        self.held = torch.zeros(rows, dtype=torch.int32, device=device)
        self.ref = torch.zeros(target.k_pages.shape[0], dtype=torch.int32, device=device)
        self.copies = torch.empty((rows, 3), dtype=torch.int32, device=device)
        self.status = torch.zeros(rows, dtype=torch.int32, device=device)                 # of the last fork
        self.refusals = torch.zeros((), dtype=torch.int64, device=device)
        self.scores = torch.zeros((n, beams), device=device)
        self.finished = torch.zeros((n, beams), dtype=torch.bool, device=device)
        self.tokens = torch.zeros((n, beams), dtype=torch.int32, device=device)           # not yet in the cache
        self.history = torch.full((n, beams, steps), end_token, dtype=torch.int32, device=device)
        self.length = torch.zeros(rows, dtype=torch.int32, device=device)                 # cached tokens of a beam
        self.place = torch.arange(beams, dtype=torch.int32, device=device).expand(n, beams)
        self.done = torch.zeros((), dtype=torch.int64, device=device)                     # steps taken

    def room(self, parent, group, keep, length):
        self.status.zero_()
        sv.kv_fork(self.t.table, self.held, self.ref, self.t.page, keep, length, parent=parent, group=group,
                   copies=self.copies, status=self.status, ws=self.t.ws)
        sv.kv_copy(self.t.k_pages, self.t.v_pages, self.copies)
        refused = (self.status & sv.ROW_ERROR_MASK) != 0       # no room for another token: these beams end here
        self.finished |= refused.view(self.n, self.beams)
        self.length.masked_fill_(refused, 0)                   # (their pages go back with the next fork)
        self.refusals += refused.sum()

    def start(self, prompts: torch.Tensor):
        """Prompts [n, length] into the first beam of every request, and its best continuations into all of them."""
        n, beams, p = self.n, self.beams, prompts.shape[1]
        first = torch.arange(n * beams, device=prompts.device) % beams == 0
        self.length.copy_(first * p)
        self.room(None, 0, torch.zeros_like(self.length), self.length)
        if int(self.refusals):
            raise RuntimeError("the pool has no pages for the prompts")
        qo = torch.zeros(n * beams + 1, dtype=torch.int32, device=prompts.device)
        qo[1:] = self.length.cumsum(0)
        logits = self.t.forward(prompts.reshape(-1), qo, self.length, p)
        one = logits.view(n, p, -1)[:, p - 1:]                                             # [n, 1, vocab]
        out = sv.beam_select(one, self.scores[:, :1].contiguous(), beams, ws=self.t.ws)
        self.follow(out)
        return one, out

    def follow(self, out):
        """The selected continuations become the beams."""
        refused = out.parents < 0                              # a request whose selection was: its beams end as they are
        parents = torch.where(refused, self.place, out.parents)
        self.tokens.copy_(out.tokens.masked_fill(refused, self.end))
        self.scores.copy_(torch.where(refused, self.scores, out.scores))
        self.finished.copy_(sv.beam_reorder(self.finished, parents))
        sv.beam_reorder(self.history, parents, out=self.history)
        self.history.scatter_(2, self.done.expand(self.n, self.beams, 1), self.tokens[..., None])
        self.finished |= self.tokens == self.end
        self.done += 1
        over = self.finished.view(-1)
        keep = sv.beam_reorder(self.length.view(self.n, self.beams), parents).view(-1).masked_fill(over, 0)
        self.length.copy_((keep + 1).masked_fill(over, 0))
        self.room(parents.view(-1), self.beams, keep, self.length)

    def step(self):
        """Append the beams' tokens, score and select.  Returns (logits [n, beams, vocab], selection)."""
        rows = self.n * self.beams
        live = ~self.finished.view(-1)
        qo = torch.zeros(rows + 1, dtype=torch.int32, device=live.device)
        qo[1:] = live.cumsum(0)
        packed = torch.zeros(rows + 1, dtype=torch.int32, device=live.device)
        packed.scatter_(0, torch.where(live, qo[:-1], rows).long(), self.tokens.view(-1))  # finished beams have no window
        logits = self.t.forward(packed[:rows], qo, self.length, 1)
        logits = logits[qo[:-1].long().clamp(max=rows - 1)].view(self.n, self.beams, -1)
        out = sv.beam_select(logits, self.scores, self.beams, finished=self.finished, end_token=self.end, ws=self.t.ws)
        self.follow(out)
        return logits, out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    sv.load(build_if_missing=True)
    prompt = 24
    target = Target(a.requests * a.beams, max_len=prompt + a.steps + 1)
    search = BeamSearch(target, a.requests, a.beams, a.steps, end_token=1)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = torch.randint(2, target.vocab, (a.requests, prompt), generator=g, device="cuda", dtype=torch.int32)
    search.start(prompts)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for s in range(1, a.steps):
        if s == 2:
            start.record()
        search.step()
    stop.record()
    torch.cuda.synchronize()
    if int(search.refusals):
        print(f"{int(search.refusals)} beams ended for want of pages")
    pages = int((search.ref > 0).sum())
    print(f"{a.requests} requests x {a.beams} beams, {a.steps} tokens: best score {float(search.scores.max()):.3f}, "
          f"{pages} pages for {int(search.held.sum())} held, {start.elapsed_time(stop) / max(a.steps - 2, 1):.3f} ms a step")


if __name__ == "__main__":
    main()
