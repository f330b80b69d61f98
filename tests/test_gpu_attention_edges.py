"""The attention operators at the edges of their promises: limits that do not limit."""
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
