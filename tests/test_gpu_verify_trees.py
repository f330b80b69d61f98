"""Verify steps of trees of drafts over a pool of pages: room, append, an accepted path moved together, the rest given back, and
the next step's logits against the dense layer on the committed tokens."""
import os
import sys

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.test_gpu_target_step import dense_logits

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.mark.parametrize("page,nodes,d", [(8, 7, 64), (16, 13, 128), (4, 23, 64)])
def test_accepted_paths_of_trees_stay_on_the_dense_layers_logits(page, nodes, d):
    from target_step import Target
    n, vocab, window = 4, 64, 2
    t = Target(n, max_len=140, vocab=vocab, hq=4, hkv=2, d=d, page=page)
    held = torch.zeros(n, dtype=torch.int32, device="cuda")
    ref = torch.zeros(t.k_pages.shape[0], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(nodes)
    draw = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)   # noqa: E731
    qo = torch.arange(0, n * nodes + 1, nodes, dtype=torch.int32, device="cuda")
    next_qo = torch.arange(0, n * window + 1, window, dtype=torch.int32, device="cuda")
    text, moved = [[] for _ in range(n)], 0
    for s in range(7):
        # a node's parent stands before it; its key is rotated for its depth
        parent = [[-1] + [int(draw(0, j, 1)) for j in range(1, nodes)] for _ in range(n)]
        depth = torch.zeros((n, nodes), dtype=torch.int32)
        for r in range(n):
            for j in range(1, nodes):
                depth[r, j] = depth[r, parent[r][j]] + 1
        tokens = draw(0, vocab, n, nodes)
        copies = sv.kv_fork(t.table, held, ref, page, t.kv_len, t.kv_len + nodes, ws=t.ws)
        assert (copies == -1).all()
        qkv = (t.embed[tokens.view(-1).long()] @ t.w_qkv).view(-1, t.hq + 2 * t.hkv, t.d)
        _, k, v = qkv.split([t.hq, t.hkv, t.hkv], dim=1)
        at = (t.kv_len[:, None] + depth.cuda()).view(-1)
        k = sv.rotary(k, at, t.freq, t.interleaved, mscale=t.mscale)
        sv.kv_append(k, v, t.k_pages, t.v_pages, t.table, qo, t.kv_len + nodes)
        # the path to some node
        paths = []
        for r in range(n):
            j, path = int(draw(0, nodes, 1)), []
            while j >= 0:
                path.append(j)
                j = parent[r][j]
            paths.append(path[::-1])
        keep = torch.full((n, nodes), -1, dtype=torch.int32)
        for r, p in enumerate(paths):
            keep[r, :len(p)] = torch.tensor(p)
            moved += sum(j != i for i, j in enumerate(p))
        count = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        sv.kv_compact(t.k_pages, t.v_pages, t.table, keep.cuda(), count, first=t.kv_len)
        t.kv_len += count
        sv.kv_fork(t.table, held, ref, page, t.kv_len, t.kv_len, ws=t.ws)
        for r, p in enumerate(paths):
            text[r] += tokens[r, p].tolist()
        assert held.tolist() == [-(-len(x) // page) for x in text]
        assert int(ref.sum()) == int(held.sum()) and int(ref.max()) <= 1
        # a window of the next step, given back as well
        nxt = draw(0, vocab, n, window)
        sv.kv_fork(t.table, held, ref, page, t.kv_len, t.kv_len + window, ws=t.ws)
        logits = t.forward(nxt.view(-1), next_qo, t.kv_len + window, window)
        for r in range(n):
            want = dense_logits(t, torch.tensor(text[r] + nxt[r].tolist(), device="cuda"))[-window:].float()
            # roundings of 2^-9 and sums in other orders, as in the decoding loop of the target step
            assert (logits[r * window:(r + 1) * window].float() - want).abs().max() <= 0.03 * want.abs().max(), (s, r)
        sv.kv_fork(t.table, held, ref, page, t.kv_len, t.kv_len, ws=t.ws)
    assert moved >= 10                              # kept tokens whose place was another
