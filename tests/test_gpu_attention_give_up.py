"""sv_paged_attention built with waits that give up after a few polls: a call that gives up says so, touches nothing but
its own rows, leaves nothing in flight and the GPU usable."""
import os
import subprocess

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.attention_cases import Batch, attend64

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
POLLS = (1, 20, 300)

SHAPES = {
    "windows": ([1, 8, 3, 16] * 12, [900, 1300, 260, 77] * 12, 16, 4, 128, 16, BF16),
    "queries by warps": ([2, 9, 25] * 8, [700, 129, 400] * 8, 10, 2, 64, 16, F16),
    "prompts": ([300, 150, 513], [700, 1150, 513], 4, 2, 128, 64, BF16),
    "prompts, heads of 64": ([300, 150, 513], [700, 150, 2513], 4, 2, 64, 32, F16),
    "one long request": ([4], [20_000], 4, 1, 128, 64, BF16),
    "short caches": ([4, 1] * 100, [300, 40] * 100, 8, 2, 64, 16, BF16),
}


@pytest.fixture(scope="module")
def libraries(tmp_path_factory):
    """The library with the tensor-core attention's waits limited to so many polls."""
    sv_build.build()
    sv.load()
    objects = [os.path.join(sv_build.BUILD_DIR, x.replace(".cu", ".o")) for x in sv_build.SOURCES]
    if not all(os.path.exists(x) for x in objects):
        sv_build.build(force=True)
    where = tmp_path_factory.mktemp("give_up")
    nvcc, source = sv_build._nvcc(), os.path.join(sv_build.CSRC, "sv_attn_tc.cu")
    jobs = []
    for n in POLLS:
        obj = str(where / f"attn{n}.o")
        jobs.append((n, obj, subprocess.Popen([nvcc, *sv_build.ARCH, *sv_build.FLAGS, f"-DSV_ATTN_WAIT_POLLS={n}", "-c",
                                               source, "-o", obj])))
    libs = {}
    for n, obj, job in jobs:
        assert job.wait() == 0
        libs[n] = str(where / f"libsv{n}.so")
        subprocess.check_call([nvcc, *sv_build.ARCH, "-shared", "-o", libs[n], obj, "-lcudart",
                               *[x for x in objects if not x.endswith("sv_attn_tc.o")]])
    return libs


@pytest.fixture(params=POLLS)
def impatient(request, libraries, monkeypatch):
    monkeypatch.setattr(sv_build, "LIB_PATH", libraries[request.param])
    monkeypatch.setattr(sv, "_lib", None)
    sv.load()
    return request.param


def guarded(shape, dtype, value, room=4096):
    """A tensor in the middle of a larger one full of `value`: (tensor, whole, its place)."""
    n = 1
    for x in shape:
        n *= x
    whole = torch.full((n + 2 * room,), value, dtype=dtype, device="cuda")
    return whole[room:room + n].view(shape), whole, slice(room, room + n)


def outside(whole, place):
    return torch.cat([whole[:place.start], whole[place.stop:]])


@pytest.mark.parametrize("name", list(SHAPES))
def test_a_call_that_gives_up_says_so_and_touches_only_its_rows(impatient, name):
    b = Batch(*SHAPES[name], seed=51, pad_tokens=3)
    q, kp, vp, table, qo, kv_len = b.gpu()
    copies = [x.clone() for x in (q, kp, vp, table, qo, kv_len)]
    ws = sv.Workspace("cuda")
    seen = set()
    for _ in range(12):
        out, whole, place = guarded(q.shape, b.dtype, 3.0)
        status = torch.zeros(b.n, dtype=torch.int32, device="cuda")
        sv.paged_attention(q, kp, vp, table, qo, kv_len, max(b.windows), out=out, status=status, ws=ws)
        torch.cuda.synchronize()
        assert len(set(status.tolist())) == 1
        seen.add(status[0].item())
        assert (out[b.qo[-1]:] == 3.0).all() and (outside(whole, place) == 3.0).all()
        for x, y in zip((q, kp, vp, table, qo, kv_len), copies):
            assert torch.equal(x.nan_to_num(7.0) if x.is_floating_point() else x,
                               y.nan_to_num(7.0) if y.is_floating_point() else y)
    assert seen <= {0, sv.ROW_TIMEOUT}
    assert impatient > 1 or seen == {sv.ROW_TIMEOUT}        # one poll is too few for any call


def test_the_next_call_is_right(libraries, monkeypatch):
    b = Batch([1, 8, 200], [900, 2300, 400], 16, 4, 128, 16, BF16, seed=52)
    out, _, tol, _ = attend64(b)
    args = b.gpu()
    with monkeypatch.context() as m:
        m.setattr(sv_build, "LIB_PATH", libraries[1])
        m.setattr(sv, "_lib", None)
        sv.load()
        ws = sv.Workspace("cuda")
        for _ in range(5):
            sv.paged_attention(*args, 200, ws=ws)
    status = torch.zeros(b.n, dtype=torch.int32, device="cuda")
    got = sv.paged_attention(*args, 200, ws=ws, status=status)          # the same workspace, on the same stream
    assert status.tolist() == [0] * b.n and ((got.out.double().cpu() - out).abs() <= tol).all()


@pytest.mark.parametrize("name", list(SHAPES))
def test_results_of_a_call_that_gives_up_are_right_or_nan(impatient, name):
    b = Batch(*SHAPES[name], seed=53, pad_tokens=2)
    want, lse, tol, tol_l = attend64(b)
    args = b.gpu()
    ws, live, missing = sv.Workspace("cuda"), b.qo[-1], 0
    for _ in range(12):
        out = torch.full(args[0].shape, 3.0, dtype=b.dtype, device="cuda")
        status = torch.zeros(b.n, dtype=torch.int32, device="cuda")
        got = sv.paged_attention(*args, max(b.windows), out=out, status=status, ws=ws)
        o, m = got.out[:live].double().cpu(), got.lse[:live].double().cpu()
        assert (o.isnan() | ((o - want[:live]).abs() <= tol[:live])).all()
        assert (m.isnan() | (m == lse[:live]) | ((m - lse[:live]).abs() <= tol_l[:live])).all()
        missing += int(o.isnan().sum())
        assert status[0].item() == sv.ROW_TIMEOUT or not (o.isnan().any() or m.isnan().any())
        quiet = sv.paged_attention(*args, max(b.windows), ws=ws)             # and without a status
        o = quiet.out[:live].double().cpu()
        assert (o.isnan() | ((o - want[:live]).abs() <= tol[:live])).all()
    assert impatient > 1 or missing
