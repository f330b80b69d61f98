"""sv.beam_select where scores and logits lie at the ends of fp32: the lowest finite score, of finished and of live beams."""
import math

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.beam_cases import score_tolerance, select64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LOWEST = torch.finfo(F32).min
# items, continuations: one launch of clusters; three with CTAs of 1,024 threads that pick; three with small CTAs
FORMS = [(5, 4), (170, 12), (170, 4)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.fixture(scope="module")
def ws():
    return sv.Workspace("cuda")


def among(logits, fill):
    """The logits on the device, `fill` on both sides of every item."""
    n, beams, vocab = logits.shape
    wide = torch.full((n + 2, beams + 2, vocab), fill, dtype=logits.dtype, device="cuda")
    view = wide[1:-1, 1:-1]
    view.copy_(logits)
    return view


def poisoned(n, n_out):
    """Outputs in which what is not written shows."""
    return sv.BeamOut(torch.full((n, n_out), -77, dtype=torch.int32, device="cuda"),
                      torch.full((n, n_out), -77, dtype=torch.int32, device="cuda"),
                      torch.full((n, n_out), math.nan, device="cuda"))


def check(logits, scores, n_out, ws, finished=None, end_token=0, view=None):
    n = len(logits)
    status = torch.zeros(n, dtype=torch.int32, device="cuda")
    got = sv.beam_select(logits.cuda() if view is None else view, scores.cuda(), n_out,
                         finished=None if finished is None else finished.cuda(), end_token=end_token,
                         out=poisoned(n, n_out), status=status, ws=ws)
    tokens, parents, want = select64(logits, scores, n_out, finished, end_token)
    assert status.tolist() == [0] * n
    assert torch.equal(got.parents.cpu(), parents)
    assert torch.equal(got.tokens.cpu(), tokens)
    # in fp32, in which a score below its lowest finite number is -inf
    s, want32 = got.scores.cpu(), want.float()
    assert ((s == want32) | ((s.double() - want).abs() <= score_tolerance(want))).all()


@pytest.mark.parametrize("n,n_out", FORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_finished_beams_of_the_lowest_score(ws, dtype, n, n_out):
    # an idle request of a batch: all of its beams finished, with the lowest score there is
    beams, vocab, end = 12, 3001, 2000
    g = torch.Generator().manual_seed(n_out)
    logits = (torch.randn((n, beams, vocab), generator=g) * 3).to(dtype)
    scores = -10.0 * torch.rand((n, beams), generator=g)
    finished = torch.zeros((n, beams), dtype=torch.bool)
    idle = [0, 1, 3, n - 1]
    finished[idle] = True
    scores[idle] = LOWEST
    scores[1] = LOWEST + 2.0 ** 104 * torch.randint(0, 4, (beams,), generator=g)
    scores[3, ::2] = -math.inf                      # and beams that are dead
    scores[3, 1::2] = LOWEST
    view = among(logits, 60.0)                      # what would come first if it were read
    view[torch.tensor(idle)] = 50.0
    check(logits, scores, min(n_out, 6), ws, finished, end, view)
    check(logits, scores, n_out, ws, finished, end, view)


@pytest.mark.parametrize("n", [2, 160])
@pytest.mark.parametrize("beams,n_out", [(16, 16), (128, 100)])
def test_idle_items_of_many_chunks(ws, n, beams, n_out):
    # more chunks than an item may list
    vocab, end = 151936 if beams == 16 else 20011, 7
    scores = torch.full((n, beams), LOWEST)
    scores[:, 1::3] += 2.0 ** 105
    row = torch.full((vocab,), math.nan, dtype=BF16, device="cuda")
    got = sv.beam_select(row.expand(n, beams, vocab), scores.cuda(), n_out, out=poisoned(n, n_out),
                         finished=torch.ones((n, beams), dtype=torch.bool, device="cuda"), end_token=end, ws=ws)
    best, parents = scores.sort(dim=-1, descending=True, stable=True)
    assert torch.equal(got.parents.cpu(), parents[:, :n_out].to(torch.int32))
    assert (got.tokens == end).all() and torch.equal(got.scores.cpu(), best[:, :n_out])


@pytest.mark.parametrize("n,n_out", FORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("down", [1.0, 1 - 2.0 ** -22, 1 - 2.0 ** -21, 1 - 2.0 ** -20, 0.5])
def test_live_beams_of_the_lowest_score(ws, dtype, n, n_out, down):
    # no logit tells in such a score: equal ones go by their place
    beams, vocab = 12, 1501
    g = torch.Generator().manual_seed(n)
    logits = (torch.randn((n, beams, vocab), generator=g) * 3).to(dtype)
    scores = -10.0 * torch.rand((n, beams), generator=g)
    scores[1:n - 1:2] = LOWEST * down
    scores[3, 2:] = -math.inf
    finished = torch.rand((n, beams), generator=g) < 0.3
    view = among(logits, 60.0)
    view[finished.cuda()] = 50.0                    # not read
    check(logits, scores, n_out, ws, finished, 9, view)
