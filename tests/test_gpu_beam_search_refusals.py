"""A search goes on where a call refuses a request: its beams end there, and nobody else's cache is written on."""
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

N, BEAMS, PAGE, VOCAB, P, STEPS = 4, 3, 8, 96, 11, 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


def searching(end):
    from beam_search import BeamSearch
    from target_step import Target
    t = Target(N * BEAMS, max_len=P + STEPS + 2, vocab=VOCAB, hq=4, hkv=2, d=64, page=PAGE)
    search = BeamSearch(t, N, BEAMS, STEPS, end)
    g = torch.Generator(device="cuda").manual_seed(6)
    prompts = torch.randint(0, VOCAB, (N, P), generator=g, device="cuda", dtype=torch.int32)
    prompts[prompts == end] = end + 1
    return t, search, prompts


def texts(search, prompts, steps):
    """Every beam's tokens, its last one included."""
    return [[prompts[i].tolist() + search.history[i, b, :steps].tolist() for b in range(BEAMS)] for i in range(N)]


def step_on_the_dense_layer(t, search, prompts, steps):
    before, live = texts(search, prompts, steps), ~search.finished.cpu()
    logits, _ = search.step()
    for i in range(N):
        for b in range(BEAMS):
            if live[i, b]:
                want = dense_logits(t, torch.tensor(before[i][b], device="cuda"))[-1].float()
                # roundings as in the search that nobody is refused in
                assert (logits[i, b].float() - want).abs().max() <= 0.03 * want.abs().max(), (steps, i, b)


def counted(search, also):
    want = also.clone()
    for row, n in zip(search.t.table.tolist(), search.held.tolist()):
        for p in row[:n]:
            want[p] += 1
    return want


@pytest.mark.parametrize("left", [0, 1, 5])
def test_beams_without_pages_end(left):
    t, search, prompts = searching(end=1)
    search.start(prompts)
    # somebody else takes all free pages but a few
    free = (search.ref == 0).nonzero().view(-1)
    taken = free[left:]
    also = torch.zeros_like(search.ref)
    also[taken] = 1
    search.ref += also
    t.k_pages[taken], t.v_pages[taken] = 7.0, -7.0
    for s in range(1, STEPS):
        over = search.finished.clone()
        step_on_the_dense_layer(t, search, prompts, s)
        assert (t.k_pages[taken] == 7.0).all() and (t.v_pages[taken] == -7.0).all()
        assert torch.equal(search.ref.cpu(), counted(search, also.cpu()))
        live = ~search.finished.view(-1)
        assert torch.equal(search.length[live], torch.full_like(search.length[live], P + s + 1))
        assert (search.length[~live] == 0).all() and search.scores.isfinite().all()
        if over.all():
            assert search.held.tolist() == [0] * (N * BEAMS)
    assert int(search.refusals) > 0


def test_prompts_without_pages_are_refused():
    t, search, prompts = searching(end=1)
    search.ref += 1
    search.ref[:3] = 0
    with pytest.raises(RuntimeError, match="pages"):
        search.start(prompts)


def test_a_request_of_nan_logits_ends():
    end = 3
    t, search, prompts = searching(end)
    prompts[1, 4] = end                             # (nobody feeds it back: a beam that has it is finished)
    t.embed[end] = float("nan")
    search.start(prompts)
    assert search.finished[1].all() and not search.finished[0].all()
    for s in range(1, STEPS):
        step_on_the_dense_layer(t, search, prompts, s)
        assert search.finished[1].all() and (search.length.view(N, BEAMS)[1] == 0).all()
        assert (search.held.view(N, BEAMS)[1] == 0).all() and search.scores.isfinite().all()
        assert (search.history[1, :, :s + 1] == end).all()
        assert torch.equal(search.ref.cpu(), counted(search, torch.zeros_like(search.ref).cpu()))
