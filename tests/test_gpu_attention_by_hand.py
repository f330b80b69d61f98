"""sv_paged_attention where values that are not finite lie in tiles that only some rows of an item see, item after item of
a CTA: rows that do not see such a value must be as if it were not there, whichever item they belong to."""
import math

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.attention_cases import U, TINY, Batch, attend64

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.fixture(scope="module")
def ws():
    return sv.Workspace("cuda")


def dense64(b, window):
    """attention_cases.attend64 for long prompts: every head's rows at once, the same bounds."""
    out = torch.zeros((b.tokens, b.hq, b.d), dtype=torch.float64)
    tol = torch.zeros_like(out)
    u, scale, grp = U[b.dtype], b.d ** -0.5, b.hq // b.hkv
    for r in range(b.n):
        n, w, t0 = b.lens[r], b.windows[r], b.qo[r]
        k, v = b.cached(r, "k").double(), b.cached(r, "v").double()
        p, j = torch.arange(n - w, n)[:, None], torch.arange(n)
        seen = (j <= p) & (j > p - window)
        for h in range(b.hq):
            q, kk, vv = b.q[t0:t0 + w, h].double(), k[:, h // grp], v[:, h // grp]
            e = torch.softmax((scale * (q @ kk.T)).masked_fill(~seen, -math.inf), -1)
            size = (scale * (q.abs() @ kk.abs().T)).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
            delta = size * (b.d + 4) * 2.0 ** -24 + 2.0 ** -21
            out[t0:t0 + w, h] = e @ vv
            tol[t0:t0 + w, h] = (u * out[t0:t0 + w, h].abs() + (u + 4 * delta + 2.0 ** -20) * (e @ vv.abs()) +
                                 TINY[b.dtype])
    return out, tol


def spoil(b, r, p, what=float("nan")):
    b.v_pages[b.table[r, p // b.page].item(), p % b.page] = what


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("hq,hkv", [(16, 16), (10, 2)])     # queries by TMA, and groups whose queries warps load
@pytest.mark.parametrize("every", [0, 128])                 # one bad value a prompt, or one in the middle of every tile
def test_items_of_two_tiles_one_after_the_other(ws, dtype, d, hq, hkv, every):
    n = 2000
    b = Batch([n] * 4, [n] * 4, hq, hkv, d, 16, dtype, seed=41)
    out, tol = dense64(b, 100)
    bad = list(range(64, n, every)) if every else [704]
    for r in range(b.n):
        for p in bad:
            spoil(b, r, p)
    i = torch.arange(n)
    sees = torch.zeros(n, dtype=torch.bool)
    for p in bad:
        sees |= (i >= p) & (i < p + 100)
    sees = sees.repeat(b.n)
    q, kp, vp, table, qo, kv_len = b.gpu()
    status = torch.zeros(b.n, dtype=torch.int32, device="cuda")
    for _ in range(10):
        got = sv.paged_attention(q, kp, vp, table, qo, kv_len, n, window=100, status=status, ws=ws).out.cpu()
        assert got[sees].isnan().all()
        diff = (got[~sees].double() - out[~sees]).abs()
        assert (diff <= tol[~sees]).all(), float((diff - tol[~sees]).nan_to_num(1e9).max())
    assert status.tolist() == [0] * b.n


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("wide", [False, True])
def test_the_last_value_of_every_request(ws, dtype, d, wide):
    # items of one to three tiles, the last one by hand, hundreds of them a call; whole items under a narrow table
    g = torch.Generator().manual_seed(42)
    n = 300
    windows = torch.randint(4, 9, (n,), generator=g).tolist()
    lens = [max(w, x) for w, x in zip(windows, torch.randint(8, 385, (n,), generator=g).tolist())]
    b = Batch(windows, lens, 16, 8, d, 16, dtype, seed=43)
    out, lse, tol, tol_l = attend64(b)
    for r in range(n):
        spoil(b, r, lens[r] - 1, float("nan") if r % 2 else float("inf"))
    clean = torch.tensor([t for r in range(n) for t in range(b.qo[r], b.qo[r + 1] - 1)])
    last = torch.tensor(b.qo[1:]) - 1
    q, kp, vp, table, qo, kv_len = b.gpu()
    if wide:
        full = torch.full((n, 600), -1, dtype=torch.int32, device="cuda")
        full[:, :table.shape[1]] = table
        table = full
    status = torch.zeros(n, dtype=torch.int32, device="cuda")
    for _ in range(40):
        got = sv.paged_attention(q, kp, vp, table, qo, kv_len, 8, status=status, ws=ws)
        o, m = got.out.cpu(), got.lse.cpu().double()
        assert not o[last].isfinite().any()
        diff = (o[clean].double() - out[clean]).abs()
        assert (diff <= tol[clean]).all(), float((diff - tol[clean]).nan_to_num(1e9).max())
        assert ((m - lse).abs() <= tol_l).all()
    assert status.tolist() == [0] * n
