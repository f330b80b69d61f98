"""The attention operators at the edges of their promises: windows of no tokens, limits that do not
limit."""
import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.attention_cases import Batch, attend64

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
