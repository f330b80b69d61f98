"""Cases of beam search and of the paged cache's pages: what is timed, and what it must equal.

* ``select``   the best continuations over all beams and the vocabulary of every request, from raw logits;
* ``reorder``  state rows follow their beams' parents, in place or into another tensor;
* ``fork``     requests take over their parents' pages, grow, shrink and give pages back (bookkeeping on the device);
* ``copy``     the pages that a fork lists are copied, all layers at once;
* ``compact``  the tokens of a request that are kept move to the front, all layers at once.

``run`` computes the plain form (elementary torch operations) or, with ``own`` set, calls the framework's operators.  The
plain form of ``select`` is in fp64, because the order of two beams' candidates hangs on the difference of their normalisers,
and fp32 normalisers of a large vocabulary are off by more than candidates lie apart.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "i32": torch.int32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4, "i32": 4}
DEV = "cuda"


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one request, the smallest call: latency only
        dict(name="select one request", op="select", dtype="bf16", n=1, beams=4, n_out=8, vocab=32000, allowed=0,
             finished=False, first=False),
        # odd sizes in fp32, some beams finished, a grammar that allows a part of the vocabulary
        dict(name="select under a grammar", op="select", dtype="f32", n=7, beams=5, n_out=10, vocab=32003, allowed=9001,
             finished=True, first=False),
        # a batch in the middle of its search
        dict(name="select a batch", op="select", dtype="bf16", n=32, beams=8, n_out=16, vocab=151936, allowed=0,
             finished=True, first=False),
        # many beams over the largest vocabulary: the read of the logits is what counts
        dict(name="select many beams", op="select", dtype="bf16", n=64, beams=16, n_out=32, vocab=248320, allowed=0,
             finished=False, first=False),
        # the token histories of a batch follow their beams
        dict(name="reorder histories", op="reorder", dtype="i32", n=32, beams_in=8, beams=8, width=1001, in_place=True),
        # recurrent states of a layer, 16 heads of 128 x 128 a beam
        dict(name="reorder states", op="reorder", dtype="f32", n=16, beams_in=8, beams=8, width=262144, in_place=True),
        # after a verify step: rejected tokens' pages go back, room for the next window
        dict(name="resize verify windows", op="fork", groups=256, beams=1, page=16, len_lo=128, len_hi=4096, window=16,
             spare=512),
        # a beam step over long contexts, whose beams share all but their last pages
        dict(name="fork long beams", op="fork", groups=16, beams=8, page=16, len_lo=16384, len_hi=131072, window=1,
             spare=4096),
        # the partly filled pages of a beam step
        dict(name="copy begun pages", op="copy", dtype="bf16", layers=4, copies=160, whole=False, hkv=8, d=128, page=16,
             heads_first=False),
        # whole pages between two regions of a pool
        dict(name="copy whole pages", op="copy", dtype="f16", layers=2, copies=1021, whole=True, hkv=8, d=128, page=16,
             heads_first=True),
        # the accepted paths of trees of drafts
        dict(name="compact accepted paths", op="compact", dtype="bf16", layers=4, n=64, window=63, keep_lo=1, keep_hi=9,
             len_lo=128, len_hi=1024, hkv=8, d=128, page=16, heads_first=False),
        # half of the tokens of long contexts are evicted
        dict(name="compact evicted contexts", op="compact", dtype="bf16", layers=1, n=4, window=16383, keep_lo=8001,
             keep_hi=8192, len_lo=1, len_hi=1, hkv=8, d=128, page=32, heads_first=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "select", "reorder", "fork", "copy", "compact"])
    if op == "select":
        beams, n, vocab = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 32]), _log(rng, 1, 64), _log(rng, 1000, 262144)
        n = max(1, min(n, 128_000_000 // (beams * vocab)))
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), n=n, beams=beams,
                    n_out=min(64, beams * rng.choice([1, 2, 2, 3])), vocab=vocab,
                    allowed=rng.choice([0, 0, 0, 3, max(4, vocab // 3)]), finished=rng.random() < 0.4,
                    first=rng.random() < 0.2)
    if op == "reorder":
        in_place, beams = rng.random() < 0.6, rng.choice([2, 3, 4, 5, 8, 16, 32])
        n, width = _log(rng, 1, 64), _log(rng, 1, 262144)
        n = max(1, min(n, 32_000_000 // (beams * width)))
        return dict(op=op, dtype=rng.choice(["bf16", "f32", "i32"]), n=n,
                    beams_in=beams if in_place else rng.choice([1, beams]), beams=beams, width=width, in_place=in_place)
    if op == "fork":
        beams = rng.choice([1, 1, 2, 4, 5, 8])
        groups, hi = max(1, _log(rng, 1, 256) // beams), _log(rng, 64, 65536)
        groups = max(1, min(groups, (1 << 22) // (beams * hi // 16 + 1)))
        return dict(op=op, groups=groups, beams=beams, page=rng.choice([16, 32, 64, 128]),
                    len_lo=max(1, hi // rng.choice([1, 4, 32])), len_hi=hi, window=rng.choice([1, 1, 8, 16, 513]),
                    spare=rng.choice([0, 64, 1000, 20000]))
    d, hkv, page = rng.choice([64, 80, 128]), rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64])
    case = dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), layers=rng.choice([1, 2, 4]), hkv=hkv, d=d, page=page,
                heads_first=rng.random() < 0.4)
    token = case["layers"] * hkv * d * SIZES[case["dtype"]] * 2
    if op == "copy":
        case.update(copies=max(1, min(_log(rng, 1, 1024), 60_000_000 // (token * page))), whole=rng.random() < 0.5)
        return case
    window = _log(rng, 2, 8192)
    hi = max(1, _log(rng, 1, window))
    case.update(n=max(1, min(_log(rng, 1, 64), 60_000_000 // (token * window))), window=window, keep_lo=max(1, hi // 4),
                keep_hi=hi, len_lo=1, len_hi=rng.choice([1, 100, 1000]))
    return case


def _spread(lo, hi, n, step):
    """n whole numbers over [lo, hi] in a fixed scattered order, even over their logarithm, the ends among them."""
    if n == 1:
        return [hi]
    f = [((i * step) % 1.0) for i in range(n)]
    f[0], f[-1] = 0.0, 1.0
    return [min(hi, max(lo, int(round(math.exp(math.log(lo) + x * (math.log(hi) - math.log(lo))))))) for x in f]


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    make = {"select": _prepare_select, "reorder": _prepare_reorder, "fork": _prepare_fork, "copy": _prepare_copy,
            "compact": _prepare_compact}[case["op"]]
    return dict(make(case, g), case=case)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _randint(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _prepare_select(case, g):
    n, beams, vocab = case["n"], case["beams"], case["vocab"]
    logits = torch.empty((n, beams, vocab), dtype=DTYPES[case["dtype"]], device=DEV)
    for i in range(n):                                          # a request at a time: no fp32 copy of the whole batch
        logits[i] = torch.randn((beams, vocab), generator=g, device=DEV) * 3.0
        if case["allowed"]:                                     # the beams of a request stand in states of one grammar
            hidden = torch.ones((beams, vocab), dtype=torch.bool, device=DEV)
            allowed = torch.rand((beams, vocab), generator=g, device=DEV).topk(min(vocab, case["allowed"]), -1).indices
            logits[i].masked_fill_(hidden.scatter_(1, allowed, False), -math.inf)
    if case["allowed"] and n > 1 and beams > 1:
        logits[-1, 0] = -math.inf                               # a beam that its grammar leaves nothing
    scores = -20.0 * _rand(g, n, beams).sort(-1).values
    if case["first"]:                                           # the first step: one beam stands for all
        scores[:, 0], scores[:, 1:] = 0.0, -math.inf
    finished = None
    if case["finished"]:
        finished = _rand(g, n, beams) < 0.25
        finished[:, 0] = False
    return dict(logits=logits, scores=scores, finished=finished, end=2)


def _parents(g, n, beams_in, beams):
    """Parents as a search has them: some beams have several children, some none; a child is often its own parent's slot."""
    drawn = _randint(g, 0, beams_in, n, beams)
    same = torch.arange(beams, device=DEV, dtype=torch.int32) % beams_in
    return torch.where(_rand(g, n, beams) < 0.4, same, drawn)


def _prepare_reorder(case, g):
    shape, dtype = (case["n"], case["beams_in"], case["width"]), DTYPES[case["dtype"]]
    state = _randint(g, 0, 100000, *shape) if dtype == torch.int32 else torch.randn(shape, generator=g, device=DEV).to(dtype)
    return dict(state=state, parents=_parents(g, case["n"], case["beams_in"], case["beams"]),
                out=None if case["in_place"] else torch.zeros((case["n"], case["beams"], case["width"]), dtype=dtype,
                                                              device=DEV))


def _fork_sizes(case):
    """(tokens a group has, columns of the table, pages of the pool)"""
    lens = _spread(case["len_lo"], case["len_hi"], case["groups"], 0.4142135624)
    page, beams, window = case["page"], case["beams"], case["window"]
    cols = -(-(max(lens) + 2 * window) // page) + 1
    shared = sum(n // page for n in lens)
    tail = -(-(page + 3 * window) // page) + 1                  # a beam's own pages, and those of a step's growth
    return lens, cols, shared + 2 * tail * beams * len(lens) + case["spare"]


def _prepare_fork(case, g):
    lens, cols, n_pages = _fork_sizes(case)
    page, beams, window, groups = case["page"], case["beams"], case["window"], case["groups"]
    lens = torch.tensor(lens, device=DEV).repeat_interleave(beams)                     # [requests]
    requests = groups * beams
    # every beam of a group shares the whole pages of the context but the last; what follows is its own
    shared = (lens // page - 1).clamp(min=0) if beams > 1 else torch.zeros_like(lens)
    room = lens + window
    held = -(-room // page)
    col = torch.arange(cols, device=DEV)
    group = torch.arange(requests, device=DEV) // beams
    first_of = torch.zeros(groups, dtype=torch.int64, device=DEV)
    first_of[1:] = shared[::beams].cumsum(0)[:-1]
    own_count = held - shared
    own_first = shared[::beams].sum() + own_count.cumsum(0) - own_count
    number = torch.where(col < shared[:, None], first_of[group][:, None] + col, own_first[:, None] + col - shared[:, None])
    order = torch.randperm(n_pages, generator=g, device=DEV)                           # pages lie anywhere in the pool
    valid = col < held[:, None]
    table = torch.where(valid, order[number.clamp(0, n_pages - 1)], 0).to(torch.int32)
    ref = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    ref.index_add_(0, table[valid].long(), torch.ones(int(valid.sum()), dtype=torch.int32, device=DEV))
    # what is kept: the context and a part of the window (the accepted one); room for the next window
    keep = (lens + (_rand(g, requests) * (window + 1)).long().clamp(max=window)).to(torch.int32)
    if beams > 1:
        keep = keep.view(groups, beams)[:, :1].expand(-1, beams).reshape(-1).contiguous()
    return dict(table=table, held=held.to(torch.int32), ref=ref, keep=keep, room=keep + window,
                parent=_parents(g, groups, beams, beams).view(-1) if beams > 1 else None)


def _pages(case, g, n_pages):
    """Key and value pages [layers, n_pages, page, heads, d], or views of heads-first storage."""
    hkv, page = case["hkv"], case["page"]
    inner = (hkv, page) if case["heads_first"] else (page, hkv)
    dims = (case["layers"], n_pages, *inner, case["d"])
    k, v = (torch.randn(dims, generator=g, device=DEV, dtype=DTYPES[case["dtype"]]) for _ in range(2))
    return (k.transpose(2, 3), v.transpose(2, 3)) if case["heads_first"] else (k, v)


def _prepare_copy(case, g):
    m = case["copies"]
    k, v = _pages(case, g, 2 * m + 5)
    order = torch.randperm(2 * m + 5, generator=g, device=DEV).to(torch.int32)
    tokens = torch.full((m,), case["page"], dtype=torch.int32, device=DEV)
    if not case["whole"]:
        tokens = torch.tensor([1 + i % (case["page"] - 1) for i in range(m)], dtype=torch.int32, device=DEV)
    return dict(k=k, v=v, copies=torch.stack([order[:m], order[m:2 * m], tokens], 1).contiguous())


def _compact_sizes(case):
    """(tokens before the window, tokens kept of it) of every request"""
    return (_spread(case["len_lo"], case["len_hi"], case["n"], 0.4142135624),
            _spread(case["keep_lo"], case["keep_hi"], case["n"], 0.6180339887))


def _prepare_compact(case, g):
    before, kept = _compact_sizes(case)
    n, page, window = case["n"], case["page"], case["window"]
    cols = -(-(max(before) + window) // page)
    per = [-(-(b + window) // page) for b in before]
    n_pages = sum(per) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    first_page = torch.tensor([sum(per[:i]) for i in range(n)], device=DEV)
    number = first_page[:, None] + torch.arange(cols, device=DEV)
    table = order[number.clamp(max=n_pages - 1)].contiguous()
    kept = torch.tensor(kept, device=DEV)
    # the kept tokens of a window: as many of its places, in order
    place = _rand(g, n, window).argsort(-1)
    width = int(case["keep_hi"])
    chosen = torch.where(torch.arange(window, device=DEV) < kept[:, None], place, window).sort(-1).values[:, :width]
    k, v = _pages(case, g, n_pages)
    return dict(k=k, v=v, table=table, first=torch.tensor(before, dtype=torch.int32, device=DEV),
                keep=chosen.to(torch.int32).contiguous(), n_keep=kept.to(torch.int32))


# ---------------------------------------------------------------------------------------------------------------
# One pass: the plain form, or the framework's operators
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"select": _plain_select, "reorder": _plain_reorder, "fork": _plain_fork, "copy": _plain_copy,
            "compact": _plain_compact}[op](state, state["case"])


def _own(state, op):
    from speculative_decoding_verification_rows_gb300 import sv

    case = state["case"]
    if op == "reorder":
        return sv.beam_reorder(state["state"], state["parents"],
                               out=state["state"] if state["out"] is None else state["out"])
    if op == "copy":
        sv.kv_copy(state["k"], state["v"], state["copies"])
        return dict(k=state["k"], v=state["v"])
    if op == "compact":
        sv.kv_compact(state["k"], state["v"], state["table"], state["keep"], state["n_keep"], first=state["first"])
        return dict(k=state["k"], v=state["v"])
    if "ws" not in state:
        state["ws"] = sv.Workspace(DEV)
    if op == "fork":
        copies = sv.kv_fork(state["table"], state["held"], state["ref"], case["page"], state["keep"], state["room"],
                            parent=state["parent"], group=case["beams"], ws=state["ws"])
        return dict(table=state["table"], held=state["held"], ref=state["ref"], copies=copies)
    out = sv.beam_select(state["logits"], state["scores"], case["n_out"], finished=state["finished"],
                         end_token=state["end"], ws=state["ws"])
    return dict(tokens=out.tokens, parents=out.parents, scores=out.scores)


def _plain_select(state, case):
    n, beams, vocab, m = case["n"], case["beams"], case["vocab"], case["n_out"]
    x, c = state["logits"].double(), state["scores"].double()
    top = x.amax(-1, keepdim=True)
    x -= torch.where(top == -math.inf, 0.0, top)
    norm = x.exp().sum(-1).log()
    x += torch.where(norm == -math.inf, -math.inf, c - norm)[..., None]
    if state["finished"] is not None:
        x.masked_fill_(state["finished"][..., None], -math.inf)
        x[..., state["end"]] = torch.where(state["finished"], c, x[..., state["end"]])
    flat = x.view(n, beams * vocab)
    last = flat.topk(m, -1).values[:, -1:]                      # the worst score that is selected; ties by the lowest index
    above, tie = flat > last, flat == last
    above |= tie & (tie.cumsum(-1, dtype=torch.int32) <= m - above.sum(-1, keepdim=True))
    at = torch.arange(beams * vocab, device=DEV, dtype=torch.int32).expand(n, -1)
    at = torch.where(above, at, beams * vocab).topk(m, -1, largest=False).values.sort(-1).values.long()
    best, order = flat.gather(1, at).sort(dim=-1, descending=True, stable=True)
    at = at.gather(1, order)
    return dict(tokens=(at % vocab).to(torch.int32), parents=(at // vocab).to(torch.int32), scores=best.float())


def _plain_reorder(state, case):
    rows = torch.arange(case["n"], device=DEV)[:, None]
    moved = state["state"][rows, state["parents"].long()]
    return (state["state"] if state["out"] is None else state["out"]).copy_(moved)


def _plain_fork(state, case):
    page, table, held, ref = case["page"], state["table"], state["held"].long(), state["ref"]
    keep, room = state["keep"].long(), state["room"].long()
    requests, cols = table.shape
    r = torch.arange(requests, device=DEV)
    parent = r if state["parent"] is None else r // case["beams"] * case["beams"] + state["parent"]
    col = torch.arange(cols, device=DEV)
    kept, want = -(-keep // page), -(-room // page)
    # references: every request gives back what it held, and takes what it keeps of its parent's
    new, had, has = table[parent].long(), col < held[:, None], col < kept[:, None]
    ref.scatter_add_(0, torch.where(had, table, 0).long().view(-1), -had.to(torch.int32).view(-1))
    ref.scatter_add_(0, torch.where(has, new, 0).view(-1), has.to(torch.int32).view(-1))
    # a begun page is written on by one request alone: of those that would, the one with the most tokens in it, if
    # nobody else reads it; the others take a copy
    begun = (keep % page != 0) & (room > keep)
    at = (keep // page).clamp(max=cols - 1)
    mine = torch.where(begun, new[r, at], 0)
    rank = (keep << 32) | (requests - r)
    writers = torch.zeros_like(ref).scatter_add_(0, mine, begun.to(torch.int32))
    best = torch.zeros(ref.shape, dtype=torch.int64, device=DEV).scatter_reduce_(0, mine, torch.where(begun, rank, 0), "amax")
    copied = begun & ~((writers[mine] == ref[mine]) & (best[mine] == rank))
    # new pages: the lowest free numbers, in order of request
    need = want - kept + copied
    first = need.cumsum(0) - need
    free = ref == 0
    pages = (~free).to(torch.int8).sort(dim=-1, stable=True).indices
    served = first + need <= free.sum()
    copied &= served
    take = lambda i: pages[i.clamp(max=pages.numel() - 1)]      # noqa: E731
    here = copied[:, None] & (col == at[:, None])
    fresh = served[:, None] & (col >= kept[:, None]) & (col < want[:, None])
    page_of = torch.where(here, take(first)[:, None], take((first + copied)[:, None] + col - kept[:, None]))
    copies = torch.stack([mine, take(first), keep % page], 1).to(torch.int32)
    copies = torch.where(copied[:, None], copies, -1)
    new = torch.where(here | fresh, page_of, new)
    ref.scatter_add_(0, mine, -copied.to(torch.int32))
    ref.scatter_add_(0, torch.where(here | fresh, page_of, 0).view(-1), (here | fresh).to(torch.int32).view(-1))
    now = torch.where(served, want, kept)
    table.copy_(torch.where(col < now[:, None], new.to(torch.int32), table))
    state["held"].copy_(now)
    return dict(table=table, held=state["held"], ref=ref, copies=copies)


def _plain_copy(state, case):
    src, dst, tokens = state["copies"].long().unbind(1)
    moved = torch.arange(case["page"], device=DEV) < tokens[:, None]
    for t in (state["k"], state["v"]):
        t[:, dst] = torch.where(moved[None, :, :, None, None], t[:, src], t[:, dst])
    return dict(k=state["k"], v=state["v"])


def _plain_compact(state, case):
    page, keep = case["page"], state["keep"].long()
    j = torch.arange(keep.shape[1], device=DEV)
    here = j < state["n_keep"][:, None]
    r = torch.arange(case["n"], device=DEV)[:, None].expand_as(keep)[here]
    src, dst = ((state["first"].long()[:, None] + x)[here] for x in (keep, j.expand_as(keep)))
    where = lambda p: (state["table"][r, p // page].long(), p % page)     # noqa: E731
    (p0, s0), (p1, s1) = where(src), where(dst)
    for t in (state["k"], state["v"]):
        t[:, p1, s1] = t[:, p0, s0]
    return dict(k=state["k"], v=state["v"])


# ---------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "select":
        # rows of live beams; a subtraction, a product, an exponential, a sum and a comparison an element
        live = case["n"] * (1 if case["first"] else case["beams"] - 0.25 * (case["beams"] - 1) * case["finished"])
        return {"bytes": int(live * case["vocab"] * SIZES[case["dtype"]]) + case["n"] * (4 * case["beams"] + 12 * case["n_out"]),
                "flops": int(5 * live * case["vocab"])}
    if op == "reorder":
        n, b, a = case["n"], case["beams"], case["beams_in"]
        stay = 0.4 + 0.6 / a if case["in_place"] else 0.0       # rows that stay where they are need not move
        same = 1.0 if case["in_place"] or a < b else 0.6 - 0.6 / a
        read = a * (1.0 - same * (1.0 - 0.6 / a) ** (b - 1)) if a > 1 else 1.0   # parents that some moved row has, each once
        row = case["width"] * SIZES[case["dtype"]]
        return {"bytes": int(n * (read + b * (1.0 - stay)) * row) + 4 * n * b, "flops": 0}
    if op == "fork":
        lens, cols, n_pages = _fork_sizes(case)
        requests = case["groups"] * case["beams"]
        moved = sum(-(-n // case["page"]) for n in lens) * case["beams"] if case["beams"] > 1 else 0
        # the counts are looked through for free pages; rows of another parent are compared with the present ones (the
        # same rows, read once), and what differs is written: a page or two a request
        return {"bytes": 4 * (n_pages + moved) + requests * (4 * 4 + 12 + 16), "flops": 0}
    token = case["layers"] * case["hkv"] * case["d"] * SIZES[case["dtype"]] * 2
    if op == "copy":
        page = case["page"]
        tokens = case["copies"] * page if case["whole"] else sum(1 + i % (page - 1) for i in range(case["copies"]))
        return {"bytes": 2 * tokens * token + 12 * case["copies"], "flops": 0}
    kept = sum(_compact_sizes(case)[1])
    return {"bytes": 2 * kept * token + 4 * kept + 8 * case["n"], "flops": 0}


# ---------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    return {"select": _select64, "reorder": _reorder64, "fork": _fork64, "copy": _copy64, "compact": _compact64}[case["op"]](
        state, case)


def _select64(state, case):
    """One request at a time: every candidate's score, all of them sorted."""
    m, vocab = case["n_out"], case["vocab"]
    tokens, parents, scores = [], [], []
    for i in range(case["n"]):
        rows = []
        for b in range(case["beams"]):
            c = float(state["scores"][i, b])
            if state["finished"] is not None and bool(state["finished"][i, b]):
                row = torch.full((vocab,), -math.inf, dtype=torch.float64, device=DEV)
                row[state["end"]] = c
            else:
                l = state["logits"][i, b].double()
                row = torch.full_like(l, -math.inf)
                if c > -math.inf and float(l.max()) > -math.inf:
                    row = torch.log_softmax(l, 0) + c
            rows.append(row)
        best, at = torch.cat(rows).sort(dim=-1, descending=True, stable=True)
        scores.append(best[:m])
        parents.append(torch.div(at[:m], vocab, rounding_mode="floor"))
        tokens.append(at[:m] - parents[-1] * vocab)
    return dict(tokens=torch.stack(tokens).to(torch.int32), parents=torch.stack(parents).to(torch.int32),
                scores=torch.stack(scores))


def _reorder64(state, case):
    parents = state["parents"].tolist()
    rows = [torch.stack([state["state"][i, p] for p in of]) for i, of in enumerate(parents)]
    out = torch.stack(rows)
    return out.double() if out.is_floating_point() else out


def _fork64(state, case):
    """Requests one after the other on the host, page by page, as the rules say it."""
    page, beams = case["page"], case["beams"]
    table, held, ref = state["table"].tolist(), state["held"].tolist(), state["ref"].tolist()
    keep, room = state["keep"].tolist(), state["room"].tolist()
    n = len(held)
    if sum(held) > 4_000_000:
        return None
    parent = list(range(n)) if state["parent"] is None else [r // beams * beams + p for r, p in enumerate(state["parent"].tolist())]
    taken = [table[parent[r]][: -(-keep[r] // page)] for r in range(n)]
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
    copier = {r for rs in writers.values() for r in rs} - stays
    free = [p for p, c in enumerate(ref) if c == 0]
    copies, first = [], 0
    for r in range(n):
        copy, more = r in copier, -(-room[r] // page) - len(taken[r])
        got = free[first: first + more + copy]
        fits = first + more + copy <= len(free)
        first += more + copy
        copies.append([-1, -1, -1])
        if fits:
            if copy:
                copies[-1] = [taken[r][-1], got[0], keep[r] % page]
                ref[taken[r][-1]] -= 1
                taken[r][-1] = got[0]
            taken[r] += got[1:] if copy else got
            for p in got:
                ref[p] += 1
    for r in range(n):
        table[r][: len(taken[r])] = taken[r]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)      # noqa: E731
    return dict(table=ints(table), held=ints([len(t) for t in taken]), ref=ints(ref), copies=ints(copies))


def _copy64(state, case):
    out = {}
    for name in "kv":
        t = state[name].double()
        for src, dst, tokens in state["copies"].tolist():
            t[:, dst, :tokens] = t[:, src, :tokens]
        out[name] = t
    return out


def _compact64(state, case):
    """A request's window as one sequence; its kept tokens in front."""
    page, out = case["page"], {name: state[name].double() for name in "kv"}
    for i, (a, n) in enumerate(zip(state["first"].tolist(), state["n_keep"].tolist())):
        pages = state["table"][i].long()
        slots = a + state["keep"][i, :n].long()
        to = torch.arange(a, a + n, device=DEV)
        for name in "kv":
            seq = out[name][:, pages[slots // page], slots % page].clone()
            out[name][:, pages[to // page], to % page] = seq
    return out
