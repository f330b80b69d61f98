"""sv.beam_select against scores in 64 bits and a full sort, and sv.beam_reorder against indexing."""
import math

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.beam_cases import score_tolerance, select64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LOWEST = {BF16: torch.finfo(BF16).min, F32: torch.finfo(F32).min}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.fixture(scope="module")
def ws():
    return sv.Workspace("cuda")


def make(n, beams, vocab, dtype, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn((n, beams, vocab), generator=g) * scale).to(dtype)
    scores = -10.0 * torch.rand((n, beams), generator=g)
    return logits, scores, g


def check(logits, scores, n_out, ws=None, finished=None, end_token=0, view=None):
    """The operator on the device against the definition; `view`: the logits as they lie on the device."""
    x = logits.cuda() if view is None else view
    status = torch.zeros(len(logits), dtype=torch.int32, device="cuda")
    got = sv.beam_select(x, scores.cuda(), n_out, finished=None if finished is None else finished.cuda(),
                         end_token=end_token, status=status, ws=ws)
    tokens, parents, want = select64(logits, scores, n_out, finished, end_token)
    assert status.tolist() == [0] * len(logits)
    assert torch.equal(got.parents.cpu(), parents)
    assert torch.equal(got.tokens.cpu(), tokens)
    s = got.scores.double().cpu()
    assert ((s == want) | ((s - want).abs() <= score_tolerance(want))).all()
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,beams,vocab,n_out", [
    (1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 5, 15), (3, 2, 33, 4), (2, 4, 1000, 8), (5, 4, 1024, 8), (2, 5, 2047, 10),
    (3, 3, 2049, 6), (1, 4, 32000, 8), (2, 8, 32003, 16), (2, 1, 70001, 5), (1, 16, 9999, 64), (2, 128, 515, 256),
    (1, 3, 524288, 9), (40, 2, 4097, 4)])
def test_the_best_of_all_beams(ws, dtype, n, beams, vocab, n_out):
    logits, scores, _ = make(n, beams, vocab, dtype, 7 * vocab + n)
    check(logits, scores, n_out, ws)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("first,step", [(0, 3), (1, 1), (3, 7), (5, 13), (7, 8)])
def test_rows_anywhere(ws, dtype, first, step):
    # a padded vocabulary, rows that begin at every boundary, items and beams the other way round
    n, beams, vocab = 3, 4, 5001
    logits, scores, _ = make(n, beams, vocab, dtype, first)
    wide = torch.full((beams, n, vocab + step + first), math.nan, dtype=dtype, device="cuda")
    view = wide[:, :, first:first + vocab].transpose(0, 1)
    view.copy_(logits)
    check(logits, scores, 8, ws, view=view)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_finished_and_dead_beams(ws, dtype):
    n, beams, vocab = 6, 5, 3001
    logits, scores, g = make(n, beams, vocab, dtype, 3)
    finished = torch.rand((n, beams), generator=g) < 0.4
    finished[2] = True                              # nothing goes on
    finished[3] = False
    scores[4, 1:] = -math.inf                       # one beam
    scores[5, 0] = -math.inf
    finished[5, 0] = True
    logits[4, 1:] = math.nan                        # rows that are not read
    logits[finished] = math.nan
    x = torch.where(logits.isnan(), 0.0, logits)
    for n_out in (1, 5, 10):
        check(x, scores, n_out, ws, finished, end_token=17, view=logits.cuda())
    check(x, scores, 10, ws, finished.to(torch.uint8), end_token=vocab - 1, view=logits.cuda())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [9, 3001])
@pytest.mark.parametrize("allowed", [0, 1, 2, 40])
def test_what_masks_leave(ws, dtype, vocab, allowed):
    n, beams, n_out = 4, 3, 12
    logits, scores, g = make(n, beams, vocab, dtype, vocab + allowed)
    hidden = torch.ones(logits.shape, dtype=torch.bool)
    hidden.scatter_(2, torch.rand(logits.shape, generator=g).topk(min(allowed, vocab), -1).indices, False)
    hidden[3, 1:] = True                            # beams without a token
    check(logits.masked_fill(hidden, -math.inf), scores, n_out, ws)
    check(logits.masked_fill(hidden, LOWEST[dtype]), scores, n_out, ws)
    check(logits.masked_fill(hidden, -1e9 if dtype is F32 else -30000.0), scores, n_out, ws)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scores_of_extreme_size(ws, dtype):
    logits, scores, _ = make(4, 4, 1500, dtype, 5)
    scores[0] -= 1e9                                # every beam as a mask would have it
    scores[1, 1] = torch.finfo(F32).min
    logits[2] += 20000.0
    logits[3] *= 1e30
    check(logits, scores, 8, ws)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("values", [1, 2, 5])
def test_rows_of_few_values(ws, dtype, values):
    # more equal candidates than a list holds: the order is by place
    n, beams, vocab = 2, 3, 70001
    _, scores, g = make(n, beams, 1, dtype, values)
    logits = torch.randint(0, values, (n, beams, vocab), generator=g).to(dtype)
    scores[0] = -1.0                                # and between beams
    check(logits, scores, 24, ws)
    check(logits[:, :, :3], scores, 9, ws)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,beams,vocab,n_out", [(50, 2, 9001, 5), (1, 64, 70001, 70), (45, 30, 40001, 3)])
def test_rows_of_one_value_in_large_calls(ws, dtype, n, beams, vocab, n_out):
    logits = torch.full((n, beams, vocab), 1.25, dtype=dtype)
    logits[n // 2, beams // 2, vocab // 2] = 1.5
    scores = torch.full((n, beams), -0.5)
    scores[0, beams - 1] = -0.25
    check(logits, scores, n_out, ws)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("beams,vocab,n_out", [(1, 32003, 64), (1, 4000, 8), (2, 30000, 256), (8, 9000, 250), (32, 2100, 40)])
@pytest.mark.parametrize("spread", [0.0, 40.0])
def test_few_rows_for_what_is_asked(ws, dtype, beams, vocab, n_out, spread):
    # fewer chunks than continuations, and beams so far apart that the bound of the best is none for them
    logits, scores, _ = make(3, beams, vocab, dtype, beams + n_out)
    scores -= spread * torch.arange(beams)
    scores[2, 1:] = -math.inf                       # the first step
    check(logits, scores, n_out, ws)
    check(logits * 40.0, scores, n_out, ws)


@pytest.mark.parametrize("n", [6, 90])                              # one launch, and three
@pytest.mark.parametrize("near", [False, True])
def test_scores_are_replaced_in_place(ws, n, near):
    # (near: every beam summed again, from the score that it had)
    beams, vocab = 6, 3001
    logits, scores, g = make(n, beams, vocab, F32, n)
    if near:
        logits[:] = logits[:, :1].clone()
        scores[:] = scores[:, :1] + 2.0 ** -20 * torch.rand(n, beams, generator=g).argsort(-1)
    tokens, parents, want = select64(logits, scores, beams)
    mine = scores.cuda()
    out = sv.BeamOut(torch.empty(n, beams, dtype=torch.int32, device="cuda"),
                     torch.empty(n, beams, dtype=torch.int32, device="cuda"), mine)
    sv.beam_select(logits.cuda(), mine, beams, out=out, ws=ws)
    assert torch.equal(out.tokens.cpu(), tokens) and torch.equal(out.parents.cpu(), parents)
    assert ((mine.double().cpu() - want).abs() <= score_tolerance(want)).all()


@pytest.mark.parametrize("n", [3, 200])
def test_one_row_for_all_beams(ws, n):
    # a search's first step: one row for all beams, all but one of them dead, or all of them alive
    logits, scores, _ = make(n, 1, 5003, BF16, n)
    first = torch.full((n, 4), -math.inf)
    first[:, 0] = 0.0
    for s in (first, -torch.arange(4.0).expand(n, 4).contiguous()):
        check(logits.expand(n, 4, 5003).contiguous(), s, 8, ws, view=logits.cuda().expand(n, 4, 5003))


@pytest.mark.parametrize("n", [2, 3])
def test_offsets_past_32_bits(ws, n):
    # beams 2^30 elements and 3 apart, items 2^32 bytes and more
    beams, vocab = 2, 5001
    logits, scores, _ = make(n, beams, vocab, BF16, n)
    step = 2 ** 30 + 3
    wide = torch.empty((n * beams - 1) * step + vocab, dtype=BF16, device="cuda")
    view = wide.as_strided((n, beams, vocab), (2 * step, step, 1))
    view.copy_(logits)
    check(logits, scores, 8, ws, view=view)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,beams,vocab,n_out", [(160, 3, 4099, 8), (700, 2, 1001, 17), (620, 3, 300, 256), (900, 1, 40, 3)])
def test_more_items_than_run_at_once(ws, dtype, n, beams, vocab, n_out):
    logits, scores, g = make(n, beams, vocab, dtype, n)
    logits[n // 2] = logits[n // 2, :1]              # equal rows, equal scores: ordered again
    scores[n // 2] = -1.0
    logits[n // 3] = -0.5                            # one value
    logits[n // 4, 0] = -math.inf
    finished = torch.rand((n, beams), generator=g) < 0.2
    check(logits, scores, n_out, ws, finished, end_token=7)


def test_equal_beams_go_by_their_number(ws):
    logits, scores, _ = make(3, 1, 5003, F32, 11)
    logits = logits.expand(3, 6, 5003).contiguous()
    scores = torch.full((3, 6), -2.5)
    scores[1, 4] = -2.4999998
    got = check(logits, scores, 18, ws)
    assert got.parents[0, :6].tolist() == [0, 1, 2, 3, 4, 5]
    assert got.parents[1, :6].tolist() == [4, 0, 1, 2, 3, 5]
    # rows of one text at different boundaries
    wide = torch.zeros((3, 6, 5004), dtype=BF16, device="cuda")
    view = wide.view(-1)[1:1 + 18 * 5003].view(3, 6, 5003)
    view.copy_(logits)
    check(logits.to(BF16), scores, 18, ws, view=view)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [4000, 50001])
@pytest.mark.parametrize("seed,n", [(0, 8), (1, 8), (2, 8), (3, 60)])       # one launch, and three
def test_beams_nearer_than_fp32_tells(ws, dtype, vocab, seed, n):
    # one row for all beams but for tokens of little mass: the sums differ by 1e-6 to 1e-9 of themselves
    beams = 6
    logits, _, g = make(n, 1, vocab, F32, seed, scale=2.0)
    logits = logits.expand(n, beams, vocab).clone()
    for i in range(n):
        mass = float(logits[i, 0].double().exp().sum())
        for b in range(1, beams):
            # a token whose mass is a part in 1e6 to 1e9 goes away
            want = math.log(mass * 10.0 ** -(6 + 3 * torch.rand((), generator=g).item()))
            at = (logits[i, b] - want).abs().argmin()
            logits[i, b, at] = -60.0
    scores = torch.full((n, beams), -3.0)
    check(logits.to(dtype), scores, 3 * beams, ws)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,beams,vocab,n_out", [(16, 52, 6, 78), (126, 52, 6, 100), (10, 40, 3001, 7), (100, 128, 12, 33)])
@pytest.mark.parametrize("finished", [False, True])
def test_many_near_beams_at_the_last_place(ws, dtype, n, beams, vocab, n_out, finished):
    # three equal candidates a beam, all beams' within fp32's rounding of their scores of one another: what belongs
    # before the last place may stand further behind it than its neighbour
    g = torch.Generator().manual_seed(vocab + n)
    logits = -1.0 - torch.rand(n, beams, vocab, generator=g)
    logits.scatter_(-1, torch.rand(n, beams, vocab, generator=g).argsort(-1)[..., :3], 2.0)
    logits = logits.to(dtype)
    x = logits.double()
    scores = (x.logsumexp(-1) - 2.0 - 4.0).float()
    ended = None
    if finished:                                    # theirs among the others' best
        ended = torch.rand(n, beams, generator=g) < 0.2
        scores = torch.where(ended, -4.0 + 2.0 ** -22 * torch.randint(-1, 2, (n, beams), generator=g), scores)
    # items in which no two scores in 64 bits are nearer than those are good to, unless they are one beam's and equal
    s = select64(logits, scores, beams * vocab, ended, 1)[2]
    d = s[:, :-1] - s[:, 1:]
    clear = ~((d > 0) & (d < 5e-12)).any(-1)
    assert clear.sum() >= n // 2
    check(logits[clear], scores[clear], n_out, ws, finished=None if ended is None else ended[clear], end_token=1)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_what_is_refused_is_refused_by_item(ws, dtype):
    n, beams, vocab = 7, 3, 2500
    logits, scores, _ = make(n, beams, vocab, dtype, 19)
    bad_l, bad_s = logits.clone(), scores.clone()
    bad_l[1, 2, 2499] = math.nan
    bad_l[2, 0, 0] = math.inf
    bad_s[4, 1] = math.nan
    bad_s[5, 2] = math.inf
    status = torch.zeros(n, dtype=torch.int32, device="cuda")
    got = sv.beam_select(bad_l.cuda(), bad_s.cuda(), 6, status=status, ws=ws)
    assert status.tolist() == [0, sv.ROW_NONFINITE, sv.ROW_NONFINITE, 0, sv.ROW_BAD_PARAM, sv.ROW_BAD_PARAM, 0]
    tokens, parents, _ = select64(logits, scores, 6)
    for i in range(n):
        if i in (0, 3, 6):
            assert torch.equal(got.tokens[i].cpu(), tokens[i]) and torch.equal(got.parents[i].cpu(), parents[i])
        else:
            assert got.tokens[i].tolist() == got.parents[i].tolist() == [-1] * 6
            assert got.scores[i].isnan().all()
    assert sv.beam_select(bad_l.cuda(), bad_s.cuda(), 6).tokens[1].tolist() == [-1] * 6      # without a status too


@pytest.mark.parametrize("n", [5, 44])                              # one launch, and three
def test_the_same_call_gives_the_same_bits_and_is_captured(n):
    logits, scores, g = make(n, 4, 20001, BF16, 23)
    logits[1, 1], scores[1, 1] = logits[1, 0], scores[1, 0]              # an item that is ordered again
    logits[2] = 1.0                                                     # and one that is picked by turns
    x, c, ws = logits.cuda(), scores.cuda(), sv.Workspace("cuda")
    want = check(logits, scores, 8, ws)
    again = sv.beam_select(x, c, 8, ws=ws)
    for name in ("tokens", "parents", "scores"):
        assert torch.equal(getattr(want, name), getattr(again, name))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = sv.beam_select(x, c, 8, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out.tokens, want.tokens)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sv.beam_select(x, c, 8, out=out, ws=ws)
    logits2, scores2, _ = make(n, 4, 20001, BF16, 24)
    for _ in range(2):
        x.copy_(logits2)
        c.copy_(scores2)
        graph.replay()
        tokens, parents, _ = select64(logits2, scores2, 8)
        assert torch.equal(out.tokens.cpu(), tokens) and torch.equal(out.parents.cpu(), parents)
        logits2, scores2, _ = make(n, 4, 20001, BF16, 25)


def test_nothing_else_is_written():
    logits, scores, _ = make(3, 2, 3000, F32, 31)
    ints = torch.full((2, 5, 4), 77, dtype=torch.int32, device="cuda")
    floats = torch.full((5, 4), 77.0, device="cuda")
    out = sv.BeamOut(ints[0, 1:4], ints[1, 1:4], floats[1:4])
    sv.beam_select(logits.cuda(), scores.cuda(), 4, out=out)
    assert (ints[:, [0, 4]] == 77).all() and (floats[[0, 4]] == 77).all() and not (ints[:, 1:4] == 77).any()
    assert sv.beam_select(logits[:0].cuda(), scores[:0].cuda(), 4).tokens.shape == (0, 4)


# ---------------------------------------------------------------------------------------------------------------
# Reordering
# ---------------------------------------------------------------------------------------------------------------
TYPES = [torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8, torch.bool, torch.complex64]


def state_of(shape, dtype, g):
    if dtype is torch.bool:
        return torch.rand(shape, generator=g) < 0.5
    if dtype.is_floating_point or dtype.is_complex:
        return torch.randn(shape, generator=g, dtype=dtype if dtype.is_complex else torch.float32).to(dtype)
    return torch.randint(0, 100, shape, generator=g).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,beams,rest", [(1, 1, (5,)), (3, 2, ()), (4, 5, (7, 3)), (2, 8, (1001,)), (3, 9, (33,)),
                                          (2, 32, (129,)), (2, 33, (65,)), (1, 128, (300,)), (2, 4, (0,))])
def test_rows_follow_their_parents(dtype, n, beams, rest):
    g = torch.Generator().manual_seed(n * beams)
    state = state_of((n, beams, *rest), dtype, g)
    parents = torch.randint(0, beams, (n, beams), generator=g, dtype=torch.int32)
    want = torch.stack([state[i, parents[i].long()] for i in range(n)])
    x = state.cuda()
    got = sv.beam_reorder(x, parents.cuda())
    assert torch.equal(got.cpu(), want) and torch.equal(x.cpu(), state)
    assert sv.beam_reorder(x, parents.cuda(), out=x) is x
    assert torch.equal(x.cpu(), want)


@pytest.mark.parametrize("beams_in,beams_out", [(1, 4), (8, 3), (3, 8), (1, 128), (40, 41)])
def test_another_number_of_beams(beams_in, beams_out):
    g = torch.Generator().manual_seed(beams_in)
    state = torch.randn((3, beams_in, 6, 50), generator=g)
    parents = torch.randint(0, beams_in, (3, beams_out), generator=g, dtype=torch.int32)
    want = torch.stack([state[i, parents[i].long()] for i in range(3)])
    assert torch.equal(sv.beam_reorder(state.cuda(), parents.cuda()).cpu(), want)


@pytest.mark.parametrize("beams", [4, 12, 48])
def test_strided_rows_and_bad_parents(beams):
    # beams outside items, rows of an odd number of bytes at odd places; what is not named is left alone
    g = torch.Generator().manual_seed(beams)
    wide = state_of((beams, 5, 77), torch.uint8, g).cuda()
    view = wide[:, 1:4, 3:70].transpose(0, 1)                      # [3, beams, 67]
    before = wide.clone()
    parents = torch.randint(0, beams, (3, beams), generator=g, dtype=torch.int32)
    parents[0, 1], parents[2, 3] = -1, beams
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    sv.beam_reorder(view, parents.cuda(), out=view, status=status)
    assert status.tolist() == [sv.ROW_BAD_LAYOUT, 0, sv.ROW_BAD_LAYOUT]
    parents[0, 1], parents[2, 3] = 1, 3                            # those stayed
    want = before.clone()
    for i in range(3):
        want[:, 1 + i, 3:70] = before[parents[i].long().cuda(), 1 + i, 3:70]
    assert torch.equal(wide, want)
    out = torch.full((3, beams, 67), 9, dtype=torch.uint8, device="cuda")
    parents[1, 2] = beams + 5
    sv.beam_reorder(view, parents.cuda(), out=out)
    assert (out[1, 2] == 9).all()


def test_a_long_row():
    # offsets past 32 bits: rows of 600 MB
    state = torch.arange(9, dtype=torch.float32, device="cuda")[:, None].expand(9, 150_000_000).contiguous().view(1, 9, -1)
    parents = torch.tensor([[8, 1, 2, 3, 4, 5, 6, 7, 0]], dtype=torch.int32, device="cuda")
    sv.beam_reorder(state, parents, out=state)
    for j, v in enumerate([8, 1, 2, 3, 4, 5, 6, 7, 0]):
        assert float(state[0, j].min()) == float(state[0, j].max()) == v
