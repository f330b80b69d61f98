"""Definitions of the beam and page operators on the host, for their tests: scores in 64 bits and a full sort; requests'
pages one after the other."""
import math

import torch


def select64(logits, scores, n_out, finished=None, end_token=0):
    """(tokens, parents, scores in 64 bits) of the n_out best continuations; logits [n, beams, vocab] on the host."""
    n, beams, vocab = logits.shape
    x = logits.double()
    top = x.amax(-1, keepdim=True)
    x = x - torch.where(top == -math.inf, 0.0, top)
    z = x.exp().sum(-1, keepdim=True)
    s = torch.where(z > 0, x - z.log() + scores.double()[..., None], -math.inf)
    if finished is not None:
        ended = torch.full((vocab,), -math.inf, dtype=torch.float64)
        for i in range(n):
            for b in range(beams):
                if finished[i, b]:
                    s[i, b] = ended
                    s[i, b, end_token] = scores[i, b].double()
    best, at = s.reshape(n, -1).sort(dim=-1, descending=True, stable=True)
    at = at[:, :n_out]
    return (at % vocab).to(torch.int32), (at // vocab).to(torch.int32), best[:, :n_out]


def score_tolerance(s):
    """Of a score in fp32: the bound on the logarithm of a row's sum, and half a step."""
    return 8e-6 + 2.0 ** -24 * torch.where(s.isfinite(), s.abs(), 0.0) + 1e-11


class Pool:
    """Requests' pages on the host: table rows, reference counts, the rules of a fork step."""

    def __init__(self, n_req, max_pages, n_pages, page, extra=None):
        self.table = torch.full((n_req, max_pages), -7, dtype=torch.int32)
        self.held = torch.zeros(n_req, dtype=torch.int32)
        self.ref = torch.zeros(n_pages, dtype=torch.int32)
        self.page = page
        if extra is not None:                       # holders outside the table
            self.ref += extra

    def gpu(self):
        return self.table.cuda(), self.held.cuda(), self.ref.cuda()

    def fork(self, keep, room, parent=None, group=0):
        """One step; returns (copies, requests without pages)."""
        n, page = len(self.held), self.page
        table, held, ref = self.table.tolist(), self.held.tolist(), self.ref.tolist()
        from_ = list(range(n)) if parent is None else [
            (r // group * group if group else 0) + int(parent[r]) for r in range(n)]
        taken = [table[from_[r]][: -(-keep[r] // page)] for r in range(n)]
        for r in range(n):
            for p in table[r][: held[r]]:
                ref[p] -= 1
        for r in range(n):
            for p in taken[r]:
                ref[p] += 1
        writers = {}
        for r in range(n):
            if keep[r] % page and room[r] > keep[r]:
                writers.setdefault(taken[r][-1], []).append(r)
        stays = {min(rs, key=lambda r: (-keep[r], r)) for p, rs in writers.items() if len(rs) == ref[p]}
        copiers = {r for rs in writers.values() for r in rs} - stays
        free = [p for p, c in enumerate(ref) if c == 0]
        copies, refused, first = [], [], 0
        for r in range(n):
            copy = r in copiers
            need = -(-room[r] // page) - len(taken[r]) + copy
            got = free[first: first + need]
            fits = need == 0 or first + need <= len(free)
            first += need
            copies.append([-1, -1, -1])
            if not fits:
                refused.append(r)
                continue
            if copy:
                copies[-1] = [taken[r][-1], got[0], keep[r] % page]
                ref[taken[r][-1]] -= 1
                taken[r][-1] = got[0]
            taken[r] += got[copy:]
            for p in got:
                ref[p] += 1
        for r in range(n):
            table[r][: len(taken[r])] = taken[r]
        ints = lambda x: torch.tensor(x, dtype=torch.int32)      # noqa: E731
        self.table, self.held, self.ref = ints(table), ints([len(t) for t in taken]), ints(ref)
        return ints(copies), refused
