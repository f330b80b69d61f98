"""sv_rotary and sv_kv_append on the GPU against the rotation in 64 bits."""
import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.attention_cases import Batch, rotate64

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
IDS = ["bf16", "f16", "f32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


def check(got, want, tol):
    diff = (got.double().cpu() - want).abs()
    bad = ~(diff <= tol)
    assert not bad.any(), f"{int(bad.sum())} off, worst {float((diff - tol).max())}"


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,d,rot", [(32, 128, 128), (5, 64, 32), (3, 80, 40), (2, 256, 128), (1, 7, 6), (7, 96, 96),
                                         (4, 128, 0)])
def test_rotation_of_part_of_the_head(dtype, interleaved, heads, d, rot):
    g = torch.Generator().manual_seed(heads * d + rot)
    tokens = 37
    x = torch.randn((tokens, heads, d), generator=g).to(dtype)
    pos = torch.randint(0, 100_000, (tokens,), generator=g, dtype=torch.int32)
    freq = sv.rotary_frequencies(rot, device="cpu")[0] if rot else torch.zeros((0, 2))
    y, tol = rotate64(x, pos, freq, interleaved, mscale=1.25)
    got = sv.rotary(x.cuda(), pos.cuda(), freq.cuda(), interleaved=interleaved, mscale=1.25)
    check(got, y, tol)


@pytest.mark.parametrize("tokens", [1, 2047, 2048, 2051])
def test_token_counts_around_the_tiles(tokens):
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn((tokens, 3, 64), generator=g).to(torch.bfloat16)
    pos = torch.arange(tokens, dtype=torch.int32)
    freq = sv.rotary_frequencies(64, device="cpu")[0]
    y, tol = rotate64(x, pos, freq)
    check(sv.rotary(x.cuda(), pos.cuda(), freq.cuda()), y, tol)


def test_angles_of_far_positions():
    pos = torch.tensor([0, 1, 131_071, 2 ** 24 - 1, 2 ** 24 + 1, 2 ** 26 + 3, 2 ** 31 - 1, 2 ** 30 + 17],
                       dtype=torch.int32)
    x = torch.randn((pos.numel(), 2, 128), generator=torch.Generator().manual_seed(1))
    freq, _ = sv.rotary_frequencies(128, device="cpu")
    y, tol = rotate64(x, pos, freq)
    # fp64 turns of the oracle: position * frequency < 2^29 turns is held to 2^-24; the kernel's low product
    # position * low < 2^29 2^-24 = 32 turns is rounded to 2^-20 turns, 6e-6 radians, above 2^24
    far = (x[:, :, :64].double() ** 2 + x[:, :, 64:].double() ** 2).sqrt().repeat(1, 1, 2)
    tol = tol + (pos >= 2 ** 24).double()[:, None, None] * far * (2.0 ** -19 * 6.2832)
    check(sv.rotary(x.cuda(), pos.cuda(), freq.cuda()), y, tol)


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    # <R x, y> = <x, R' y> for the transposed map, and differences of the scalar map along random directions
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn((19, 4, 64), generator=g) for _ in range(2))
    pos = torch.randint(0, 4096, (19,), generator=g, dtype=torch.int32)
    freq = sv.rotary_frequencies(32, device="cpu")[0]
    dx, tol = rotate64(dy, pos, freq, interleaved, inverse=True, mscale=1.3)
    got = sv.rotary(dy.cuda(), pos.cuda(), freq.cuda(), interleaved=interleaved, inverse=True, mscale=1.3)
    check(got, dx, tol)
    f = lambda z: float((rotate64(z, pos, freq, interleaved, mscale=1.3)[0] * dy.double()).sum())   # noqa: E731
    for k in range(3):
        step = torch.randn(x.shape, generator=g, dtype=torch.float64)
        eps = 1e-3
        slope = (f(x.double() + eps * step) - f(x.double() - eps * step)) / (2 * eps)   # exact: the map is linear
        along = float((got.double().cpu() * step).sum())
        assert abs(slope - along) <= float((tol * step.abs()).sum()) + 1e-9 * abs(slope) + 1e-9


def test_in_place_and_strided_rows():
    g = torch.Generator().manual_seed(4)
    packed = torch.randn((23, 10, 64), generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 5000, (23,), generator=g, dtype=torch.int32)
    freq = sv.rotary_frequencies(32, device="cpu")[0]
    y, tol = rotate64(packed[:, 2:7], pos, freq)
    dev = packed.cuda()
    view = dev[:, 2:7]
    assert sv.rotary(view, pos.cuda(), freq.cuda(), out=view) is view
    check(view, y, tol)
    assert torch.equal(dev[:, :2].cpu(), packed[:, :2]) and torch.equal(dev[:, 7:].cpu(), packed[:, 7:])
    # rows that start off 16-byte boundaries, heads apart by an odd stride
    odd = torch.zeros(23 * 333 + 1, dtype=torch.bfloat16)
    strided = torch.as_strided(odd, (23, 5, 64), (333, 65, 1), 1)
    strided.copy_(packed[:, 2:7])
    dev = odd.cuda()
    got = sv.rotary(torch.as_strided(dev, (23, 5, 64), (333, 65, 1), 1), pos.cuda(), freq.cuda())
    check(got, y, tol)


def test_no_tokens():
    freq = sv.rotary_frequencies(64)[0]
    x = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert sv.rotary(x, torch.empty(0, dtype=torch.int32, device="cuda"), freq).shape == (0, 4, 64)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def appended(b, k, v, freq, interleaved, mscale, start_k, start_v):
    """The pages after the append and the bound on the keys, in 64 bits (garbage slots stay as they are)."""
    pos = torch.tensor([b.lens[r] - b.windows[r] + i for r in range(b.n) for i in range(b.windows[r])],
                       dtype=torch.int32)
    live = b.qo[-1]
    turned, tol = (k[:live].double(), torch.zeros_like(k[:live], dtype=torch.float64)) if freq is None else \
        rotate64(k[:live], pos, freq, interleaved, mscale=mscale)
    want_k, want_v, tol_k = start_k.double().clone(), start_v.double().clone(), torch.zeros_like(start_k, dtype=torch.float64)
    t = 0
    for r in range(b.n):
        for i in range(b.windows[r]):
            p = b.lens[r] - b.windows[r] + i
            if p >= 0:
                page, slot = b.table[r, p // b.page].item(), p % b.page
                want_k[page, slot], want_v[page, slot], tol_k[page, slot] = turned[t], v[t].double(), tol[t]
            t += 1
    return want_k, want_v, tol_k, pos


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("windows,lens,hq,hkv,d,rot,page,interleaved", [
    ([1], [1], 4, 1, 64, 64, 16, False),
    ([1, 1, 1], [5, 16, 17], 14, 2, 64, 32, 16, True),
    ([3, 0, 8, 1, 16], [9, 40, 8, 129, 300], 8, 2, 128, 128, 32, False),
    ([5, 2], [5, 33], 6, 3, 80, 40, 7, True),
    ([2, 700, 1411], [2, 900, 1500], 4, 2, 32, 32, 64, False),
    ([4, 3], [2, 0], 2, 1, 64, 64, 16, False),             # windows longer than the cache: early tokens have no place
])
def test_append_rotates_and_places(dtype, heads_first, windows, lens, hq, hkv, d, rot, page, interleaved):
    b = Batch(windows, lens, hq, hkv, d, page, dtype, seed=len(windows) + d, heads_first=heads_first, garbage=7.0,
              pad_tokens=2)
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn((b.tokens, hkv, d), generator=g).to(dtype) for _ in range(2))
    freq = sv.rotary_frequencies(rot, device="cpu")[0]
    want_k, want_v, tol_k, pos = appended(b, k, v, freq, interleaved, 1.1, b.k_pages, b.v_pages)
    q, kp, vp, table, qo, kv_len = b.gpu(heads_first)
    status = torch.zeros(b.n, dtype=torch.int32, device="cuda")
    q_out = torch.full(q.shape, 5.0, dtype=dtype, device="cuda")
    got = sv.kv_append(k.cuda(), v.cuda(), kp, vp, table, qo, kv_len, freq.cuda(), interleaved, 1.1, q=q, q_out=q_out,
                       status=status)
    check(kp, want_k, tol_k)
    check(vp, want_v, torch.zeros_like(want_v))
    live = b.qo[-1]
    y, tol = rotate64(b.q[:live], pos, freq, interleaved, mscale=1.1)
    check(got[:live], y, tol)
    assert (got[live:] == 5.0).all()                        # padding tokens are not written
    short = [int(w > n) * sv.ROW_BAD_LAYOUT for w, n in zip(windows, lens)]
    assert status.tolist() == short


def test_append_without_rotation_or_queries_is_a_copy():
    b = Batch([3, 5], [10, 21], 4, 2, 64, 16, torch.float16, garbage=0.0)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn((8, 2, 64), generator=g).to(torch.float16) for _ in range(2))
    want_k, want_v, tol, _ = appended(b, k, v, None, False, 1.0, b.k_pages, b.v_pages)
    q, kp, vp, table, qo, kv_len = b.gpu()
    assert sv.kv_append(k.cuda(), v.cuda(), kp, vp, table, qo, kv_len) is None
    assert torch.equal(kp.double().cpu(), want_k) and torch.equal(vp.double().cpu(), want_v)


def test_append_refuses_bad_pages_and_lengths_without_touching_anything():
    b = Batch([2, 2, 2, 2], [20, 20, 20, 20], 4, 2, 64, 16, torch.bfloat16, garbage=0.0)
    q, kp, vp, table, qo, kv_len = b.gpu()
    table[0, 1] = b.n_pages                                # past the pages
    table[1, 1] = -1
    kv_len[2] = 16 * table.shape[1] + 2                    # past the table
    before_k, before_v = kp.clone(), vp.clone()
    k = torch.ones((8, 2, 64), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    sv.kv_append(k, k, kp, vp, table, qo, kv_len, status=status)
    assert status.tolist() == [sv.ROW_BAD_LAYOUT] * 3 + [0]
    page = b.table[3, 1].item()
    changed = (kp != before_k).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [page] and torch.equal(kp[page, 2:4], k[6:8]) and torch.equal(vp[page, 2:4], k[6:8])
    assert torch.equal(vp[:page], before_v[:page]) and torch.equal(vp[page + 1:], before_v[page + 1:])


def test_append_in_place_queries_on_another_stream_and_in_a_graph():
    b = Batch([4, 4], [40, 17], 8, 2, 128, 16, torch.bfloat16)
    freq = sv.rotary_frequencies(128)[0]
    g = torch.Generator().manual_seed(5)
    k = torch.randn((8, 2, 128), generator=g).to(torch.bfloat16).cuda()
    q, kp, vp, table, qo, kv_len = b.gpu()
    want = sv.kv_append(k, k, kp.clone(), vp.clone(), table, qo, kv_len, freq, q=q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    q2 = q.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        assert sv.kv_append(k, k, kp, vp, table, qo, kv_len, freq, q=q2, q_out=q2) is q2
    side.synchronize()
    assert torch.equal(q2, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(q)
    with torch.cuda.graph(graph):
        sv.kv_append(k, k, kp, vp, table, qo, kv_len, freq, q=q, q_out=out)
    kv_len.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    want2 = sv.kv_append(k, k, kp, vp, table, qo, kv_len, freq, q=q)
    assert torch.equal(out, want2) and not torch.equal(out, want)
