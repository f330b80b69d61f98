"""The attention operators at the edges of their promises: windows of no tokens, tokens of no window, broken
bounds, limits that do not limit."""
import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.attention_cases import Batch, attend64, rotate64

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
KERNELS = [(BF16, 128), (F16, 64), (F32, 64), (BF16, 96)]     # tensor cores, and the kernel that takes every layout


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.fixture(scope="module")
def ws():
    return sv.Workspace("cuda")


@pytest.mark.parametrize("dtype,d", KERNELS)
@pytest.mark.parametrize("hq,hkv", [(4, 2), (10, 2)])
def test_no_window_is_longer_than_nothing(ws, dtype, d, hq, hkv):
    b = Batch([0, 0, 0], [40, 0, 300], hq, hkv, d, 16, dtype, pad_tokens=5)
    q, kp, vp, table, qo, kv_len = b.gpu()
    out = torch.full_like(q, 2.0)
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    sv.paged_attention(q, kp, vp, table, qo, kv_len, max(b.windows), out=out, status=status, ws=ws)
    assert (out == 2.0).all() and status.tolist() == [0, 0, 0]


@pytest.mark.parametrize("dtype,d", KERNELS)
def test_windows_longer_than_nothing_are_refused(ws, dtype, d):
    b = Batch([0, 3, 1], [40, 9, 30], 4, 2, d, 16, dtype)
    q, kp, vp, table, qo, kv_len = b.gpu()
    out = torch.full_like(q, 2.0)
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    sv.paged_attention(q, kp, vp, table, qo, kv_len, 0, out=out, status=status, ws=ws)
    assert (out == 2.0).all() and status.tolist() == [0, sv.ROW_BAD_LAYOUT, sv.ROW_BAD_LAYOUT]


@pytest.mark.parametrize("dtype,d", KERNELS)
def test_tokens_before_the_first_window_are_nobodys(ws, dtype, d):
    # the last requests of a batch, over the token axis of all of them
    b = Batch([5, 2, 7], [50, 33, 130], 4, 2, d, 16, dtype, seed=61, pad_tokens=2)
    want, _, tol, _ = attend64(b)
    q, kp, vp, table, qo, kv_len = b.gpu()
    out = torch.full_like(q, 2.0)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    sv.paged_attention(q, kp, vp, table[1:], qo[1:], kv_len[1:], 7, out=out, status=status, ws=ws)
    assert (out[:5] == 2.0).all() and (out[14:] == 2.0).all()
    assert ((out.double().cpu() - want).abs() <= tol)[5:14].all()
    assert status.tolist() == [0, 0]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,hq", [(16, 4), (2600, 4), (2600, 40), (2601, 40)])     # one token a CTA, and several
def test_append_leaves_tokens_before_the_first_window_alone(dtype, tokens, hq):
    b = Batch([tokens - 9, 2, 7], [tokens, 33, 130], hq, 2, 64, 16, dtype, seed=62, pad_tokens=2, garbage=0.0)
    first = tokens - 9
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((b.tokens, 2, 64), generator=g).to(dtype) for _ in range(2))
    freq = sv.rotary_frequencies(64, device="cpu")[0]
    q, kp, vp, table, qo, kv_len = b.gpu()
    before_k, before_v = kp.clone(), vp.clone()
    out = torch.full_like(q, 2.0)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    sv.kv_append(k.cuda(), v.cuda(), kp, vp, table[1:], qo[1:], kv_len[1:], freq.cuda(), q=q, q_out=out, status=status)
    assert status.tolist() == [0, 0]
    assert (out[:first] == 2.0).all() and (out[first + 9:] == 2.0).all()
    pos = torch.tensor([31, 32] + list(range(123, 130)), dtype=torch.int32)
    y, tol = rotate64(b.q[first:first + 9], pos, freq)
    assert ((out[first:first + 9].double().cpu() - y).abs() <= tol).all()
    rows = [(r, p) for r, lo, hi in ((1, 31, 33), (2, 123, 130)) for p in range(lo, hi)]
    for i, (r, p) in enumerate(rows):
        at = b.table[r, p // 16].item(), p % 16
        assert torch.equal(vp[at].cpu(), v[first + i])
        before_k[at], before_v[at] = kp[at], vp[at]
    assert torch.equal(kp, before_k) and torch.equal(vp, before_v)      # and nothing else


@pytest.mark.parametrize("dtype,d", KERNELS)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
def test_a_window_of_any_size_over_rows_before_the_cache(ws, dtype, d, window):
    # rows at negative positions, which a window that is longer than any cache does not limit
    b = Batch([6, 200, 3], [2, 150, 40], 4, 2, d, 16, dtype, seed=63)
    q, kp, vp, table, qo, kv_len = b.gpu()
    for full in (True, False):
        want, lse, tol, tol_l = attend64(b, full=full)
        got = sv.paged_attention(q, kp, vp, table, qo, kv_len, 200, window=window, full=full, ws=ws)
        assert ((got.out.double().cpu() - want).abs() <= tol).all()
        m = got.lse.double().cpu()
        assert ((m == lse) | ((m - lse).abs() <= tol_l)).all()


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
def test_windows_that_end_before_they_begin(ws, dtype, d):
    # lengths that do not fit an int, under a promise that limits nothing
    b = Batch([5, 4, 3], [50, 33, 130], 4, 2, d, 16, dtype, seed=64)
    want, _, tol, _ = attend64(b)
    q, kp, vp, table, qo, kv_len = b.gpu()
    qo[2] = -2 ** 31
    out = torch.full_like(q, 2.0)
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    sv.paged_attention(q, kp, vp, table, qo, kv_len, 2 ** 31 - 1, out=out, status=status, ws=ws)
    assert status.tolist() == [0, sv.ROW_BAD_LAYOUT, sv.ROW_BAD_LAYOUT]
    assert ((out.double().cpu() - want).abs() <= tol)[:5].all() and (out[5:] == 2.0).all()


@pytest.mark.parametrize("dtype,d", KERNELS)
@pytest.mark.parametrize("broken", [-1, -2 ** 31, 3, 100])
def test_a_broken_bound_is_its_two_windows_business(ws, dtype, d, broken):
    # the end of one window and the start of the next; the requests around them are not affected
    b = Batch([5, 4, 3, 6], [50, 33, 130, 20], 4, 2, d, 16, dtype, seed=65)
    want, _, tol, _ = attend64(b)
    q, kp, vp, table, qo, kv_len = b.gpu()
    qo[2] = broken
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = sv.paged_attention(q, kp, vp, table, qo, kv_len, 6, status=status, ws=ws).out.double().cpu()
    bad = sv.ROW_BAD_LAYOUT
    assert status.tolist() == [0, bad, bad, 0]
    for lo, hi in ((0, 5), (12, 18)):
        assert ((out - want).abs() <= tol)[lo:hi].all()
    # append: the good requests' keys reach the cache; window [3, 12) is one that append takes
    kp2, vp2 = torch.zeros_like(kp), torch.zeros_like(vp)
    k = torch.randn((b.tokens, 2, d), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    status.zero_()
    sv.kv_append(k, k, kp2, vp2, table, qo, kv_len, status=status)
    assert status.tolist() == [0, bad, 0 if broken == 3 else bad, 0]
    for r, lo in ((0, 0), (3, 12)):
        for i in range(b.windows[r]):
            p = b.lens[r] - b.windows[r] + i
            assert torch.equal(kp2[b.table[r, p // 16].item(), p % 16], k[lo + i])
