"""sv_rotary at positions past 2^24, to the bound that holds for near ones."""
import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.attention_cases import rotate64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("freq", [sv.rotary_frequencies(128, device="cpu")[0],
                                  sv.rotary_frequencies(128, base=500000.0, scaling="yarn", factor=8.0,
                                                        original_len=8192, device="cpu")[0]], ids=["plain", "yarn"])
def test_angles_of_any_position(inverse, freq):
    # The angle is promised to 4e-7 turns (2.5e-6 radians); the fp64 oracle's own turns are good to 2^29 2^-53 = 2^-24.
    # Sine, cosine and products add 6e-7 of the pair's length as for near positions: 3.5e-6 with the oracle's 4e-7.
    g = torch.Generator().manual_seed(71)
    far = torch.randint(2 ** 24, 2 ** 31 - 1, (4000,), generator=g)
    edge = torch.tensor([2 ** 24 - 1, 2 ** 24, 2 ** 24 + 1, 2 ** 25 + 1, 2 ** 26 + 3, 2 ** 30 + 65, 2 ** 31 - 1, 2 ** 31 - 64,
                         2 ** 31 - 65, 2 ** 31 - 127])
    pos = torch.cat([far, edge]).to(torch.int32)
    x = torch.randn((pos.numel(), 1, 128), generator=g)
    y, tol = rotate64(x, pos, freq, inverse=inverse)
    length = (x[:, :, :64].double() ** 2 + x[:, :, 64:].double() ** 2).sqrt().repeat(1, 1, 2)
    got = sv.rotary(x.cuda(), pos.cuda(), freq.cuda(), inverse=inverse).double().cpu()
    worst = float(((got - y).abs() / length).max())
    assert worst <= 3.5e-6, worst
