"""The beam and page operators together: a search over shared pages, and verify steps that give pages back, against the same
layer recomputed from the tokens alone."""
import os
import subprocess
import sys

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.beam_cases import select64
from tests.test_gpu_target_step import dense_logits

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


def counts_are_the_tables(table, held, ref):
    want = torch.zeros_like(ref)
    for row, n in zip(table.tolist(), held.tolist()):
        for p in row[:n]:
            want[p] += 1
    assert torch.equal(ref, want)


@pytest.mark.parametrize("beams,d,page,end", [(4, 64, 16, 1), (3, 128, 8, 5), (1, 64, 16, 9)])
def test_a_search_stays_on_the_dense_layers_logits(beams, d, page, end):
    from beam_search import BeamSearch
    from target_step import Target
    n, steps, p, vocab = 3, 14, 11, 96
    t = Target(n * beams, max_len=p + steps + 2, vocab=vocab, hq=4, hkv=2, d=d, page=page)
    search = BeamSearch(t, n, beams, steps, end)
    g = torch.Generator(device="cuda").manual_seed(beams)
    prompts = torch.randint(0, vocab, (n, p), generator=g, device="cuda", dtype=torch.int32)
    text = [[prompts[i].tolist()] * beams for i in range(n)]       # of every beam, its last token included
    scores, finished = torch.zeros((n, beams)), torch.zeros((n, beams), dtype=torch.bool)
    ended = 0
    for s in range(steps):
        logits, out = search.start(prompts) if s == 0 else search.step()
        width = logits.shape[1]
        for i in range(n):
            for b in range(width):
                if finished[i, b]:
                    continue
                want = dense_logits(t, torch.tensor(text[i][b], device="cuda"))[-1].float()
                # as in the decoding loop of the target step: sums in other orders, roundings of 2^-9 behind them
                assert (logits[i, b].float() - want).abs().max() <= 0.03 * want.abs().max()
        tokens, parents, _ = select64(logits.cpu(), scores[:, :width], beams, finished[:, :width], end)
        assert torch.equal(out.tokens.cpu(), tokens) and torch.equal(out.parents.cpu(), parents)
        scores = out.scores.cpu()
        finished = finished.gather(1, parents.long()) | (tokens == end)
        text = [[text[i][int(parents[i, b])] + [int(tokens[i, b])] for b in range(beams)] for i in range(n)]
        ended += int((tokens == end).sum())
        assert torch.equal(search.finished.cpu(), finished)
        for i in range(n):
            for b in range(beams):
                assert search.history[i, b, :s + 1].tolist() == text[i][b][p:]
        assert int(search.status.max()) == 0
        counts_are_the_tables(t.table.cpu(), search.held.cpu(), search.ref.cpu())
        lens = [0 if finished.view(-1)[r] else p + s + 1 for r in range(n * beams)]
        assert search.length.tolist() == lens and search.held.tolist() == [-(-x // page) for x in lens]
    if beams > 1:
        assert int((search.ref > 1).sum()) > 0 or ended            # beams share what they have in common


def test_a_step_is_captured_in_a_graph():
    from beam_search import BeamSearch
    from target_step import Target
    n, beams, steps = 4, 4, 12

    def make():
        t = Target(n * beams, max_len=40, vocab=128, hq=4, hkv=2, d=64)
        search = BeamSearch(t, n, beams, steps, 3)
        g = torch.Generator(device="cuda").manual_seed(2)
        search.start(torch.randint(0, 128, (n, 9), generator=g, device="cuda", dtype=torch.int32))
        search.step()
        return search

    eager, search = make(), make()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        search.step()                                              # recorded, not run
    for s in range(2, steps):
        graph.replay()
        eager.step()
    for name in ("history", "scores", "finished", "held", "ref", "length"):
        assert torch.equal(getattr(search, name), getattr(eager, name)), name


@pytest.mark.parametrize("page", [8, 16])
def test_verify_steps_that_give_pages_back(page):
    """Windows of drafts with room from the pool, their rejected part given back after every step, and an accepted path of a
    tree moved together: the cache stays that of the committed tokens."""
    from target_step import Target
    n, K, vocab = 4, 5, 64
    t = Target(n, max_len=90, K=K, vocab=vocab, hq=4, hkv=2, d=64, page=page)
    held = torch.zeros(n, dtype=torch.int32, device="cuda")
    ref = torch.zeros(t.k_pages.shape[0], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(page)
    zero = torch.zeros(n, dtype=torch.int32, device="cuda")
    qo = torch.arange(0, n * (K + 1) + 1, K + 1, dtype=torch.int32, device="cuda")
    text = [[] for _ in range(n)]
    for s in range(8):
        window = torch.randint(0, vocab, (n, K + 1), generator=g, device="cuda", dtype=torch.int32)
        lens = t.kv_len + K + 1
        copies = sv.kv_fork(t.table, held, ref, page, t.kv_len, lens, ws=t.ws)
        assert (copies == -1).all()                                # nobody shares a page
        logits = t.forward(window.view(-1), qo, lens, K + 1)
        for r in range(n):
            ids = torch.tensor(text[r] + window[r].tolist(), device="cuda")
            want = dense_logits(t, ids)[-(K + 1):].float()
            assert (logits[r * (K + 1):(r + 1) * (K + 1)].float() - want).abs().max() <= 0.03 * want.abs().max()
        # a path of one token or more, beginning with the window's first: kept as far as it is the window's beginning (its
        # keys stand at their positions), and always in place afterwards
        count = torch.randint(1, K + 2, (n,), generator=g, device="cuda", dtype=torch.int32)
        keep = torch.arange(K + 1, device="cuda", dtype=torch.int32).expand(n, -1).contiguous()
        sv.kv_compact(t.k_pages, t.v_pages, t.table, keep, count, first=t.kv_len)
        t.kv_len += count
        sv.kv_fork(t.table, held, ref, page, t.kv_len, t.kv_len, ws=t.ws)
        text = [text[r] + window[r, :int(count[r])].tolist() for r in range(n)]
        assert held.tolist() == [-(-len(x) // page) for x in text]
        counts_are_the_tables(t.table.cpu(), held.cpu(), ref.cpu())
    sv.kv_fork(t.table, held, ref, page, zero, zero, ws=t.ws)
    assert int(ref.max()) == 0 and held.tolist() == [0] * n


def test_an_accepted_path_of_a_tree():
    """A tree of drafts: every node at its depth's position, the accepted path's keys and values moved to the front of the
    window; attention over the compacted cache is that over the path alone."""
    g = torch.Generator(device="cuda").manual_seed(4)
    n, page, hkv, hq, d, before, nodes = 3, 16, 2, 4, 64, 21, 13
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)      # noqa: E731
    kp, vp = rand(12, page, hkv, d), rand(12, page, hkv, d)
    table = torch.randperm(12, generator=g, device="cuda").to(torch.int32).view(n, 4)
    depth = torch.tensor([0, 1, 1, 1, 2, 2, 2, 3, 3, 3, 4, 4, 4], dtype=torch.int32, device="cuda")
    paths = [[0, 2, 5, 9, 11], [0, 1], [0, 3, 6]]
    freq = sv.rotary_frequencies(d)[0]
    k, v = rand(n, nodes, hkv, d), rand(n, nodes, hkv, d)
    turned = torch.stack([sv.rotary(k[i], before + depth, freq) for i in range(n)])
    qo = torch.arange(0, n * nodes + 1, nodes, dtype=torch.int32, device="cuda")
    lens = torch.full((n,), before + nodes, dtype=torch.int32, device="cuda")
    sv.kv_append(turned.view(-1, hkv, d), v.view(-1, hkv, d), kp, vp, table, qo, lens)
    alone = kp.clone(), vp.clone()
    keep = torch.full((n, 5), -1, dtype=torch.int32, device="cuda")
    for i, p in enumerate(paths):
        keep[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
    count = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
    first = torch.full((n,), before, dtype=torch.int32, device="cuda")
    sv.kv_compact(kp, vp, table, keep, count, first=first)
    for i, p in enumerate(paths):                                  # the path appended on its own
        one = torch.tensor([0, len(p)], dtype=torch.int32, device="cuda")
        sv.kv_append(turned[i, p].contiguous(), v[i, p].contiguous(), *alone, table[i:i + 1], one, first[:1] + len(p))
    q = rand(n, hq, d)
    single = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    got = sv.paged_attention(q, kp, vp, table, single, before + count, 1).out
    want = sv.paged_attention(q, *alone, table, single, before + count, 1).out
    assert torch.equal(got, want)


def test_the_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "beam_search.py"), "--requests", "4", "--steps", "8"],
                       capture_output=True, text=True, timeout=200)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "pages for" in r.stdout
