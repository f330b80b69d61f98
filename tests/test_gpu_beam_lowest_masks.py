"""sv.beam_select where a low score and a masked token's logit add up to less than fp32 holds: every output place is written,
in the order of the scores in 64 bits."""
import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.test_gpu_beam_extremes import BF16, F32, FORMS, LOWEST, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.fixture(scope="module")
def ws():
    return sv.Workspace("cuda")


@pytest.mark.parametrize("n,n_out", FORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("beams,vocab", [(1, 40), (3, 1501)])
@pytest.mark.parametrize("down", [1.0, 1 - 2.0 ** -21, 0.5, 1e-3])
def test_the_lowest_scores_under_masks_of_the_lowest_value(ws, dtype, n, n_out, beams, vocab, down):
    # two tokens are allowed a beam, more are asked for
    g = torch.Generator().manual_seed(n + beams)
    logits = torch.full((n, beams, vocab), torch.finfo(dtype).min, dtype=dtype)
    at = torch.rand((n, beams, vocab), generator=g).topk(2, -1).indices
    logits.scatter_(2, at, torch.randn((n, beams, 2), generator=g).to(dtype))
    scores = torch.full((n, beams), LOWEST * down)
    scores[::3, 0] = -1.0                           # one ordinary beam before the others
    finished = torch.zeros((n, beams), dtype=torch.bool)
    finished[::2, beams - 1] = True
    check(logits, scores, n_out, ws)
    check(logits, scores, n_out, ws, finished, vocab - 1)


@pytest.mark.parametrize("n,n_out", FORMS)
@pytest.mark.parametrize("down", [0.0, 0.3, 1.0])
def test_logits_that_fill_fp32(ws, n, n_out, down):
    # differences of logits past fp32's range
    beams, vocab = 4, 1203
    g = torch.Generator().manual_seed(n)
    logits = (torch.randn((n, beams, vocab), generator=g) * 1e38).clamp(min=LOWEST, max=-LOWEST)
    scores = LOWEST * down * torch.rand((n, beams), generator=g)
    check(logits, scores, n_out, ws)
    # and a row whose best are few
    logits[:, :, 3:] = LOWEST
    check(logits, scores, n_out, ws)
