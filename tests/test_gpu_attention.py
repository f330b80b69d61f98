"""sv_paged_attention on the GPU against attention in 64 bits."""
import math

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.attention_cases import Batch, attend64

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.fixture(scope="module")
def ws():
    return sv.Workspace("cuda")


def run_and_check(b, ws, heads_first=False, window=0, full=False, scale=None, max_window=None, rows=None):
    out, lse, tol, tol_l = attend64(b, scale, window, full)
    q, kp, vp, table, qo, kv_len = b.gpu(heads_first)
    status = torch.zeros(b.n, dtype=torch.int32, device="cuda")
    dest = torch.full(q.shape, 3.0, dtype=b.dtype, device="cuda")
    got = sv.paged_attention(q, kp, vp, table, qo, kv_len, max(b.windows) if max_window is None else max_window,
                             scale=scale, window=window, full=full, out=dest, status=status, ws=ws)
    live = b.qo[-1]
    sel = slice(0, live) if rows is None else rows
    diff = (got.out.double().cpu() - out).abs()[sel]
    bad = ~(diff <= tol[sel])
    assert not bad.any(), f"{int(bad.sum())} outputs off, worst over bound {float((diff - tol[sel]).nan_to_num(1e9).max())}"
    g, w = got.lse.double().cpu()[sel], lse[sel]
    empty = w == -math.inf
    assert torch.equal(g == -math.inf, empty)
    assert (~empty).sum() == 0 or ((g - w).abs()[~empty] <= tol_l[sel][~empty]).all()
    assert (got.out[live:] == 3.0).all()
    assert status.tolist() == [0] * b.n
    return got


SHAPES = [
    # windows, lens, hq, hkv, d, page
    ([1], [1], 2, 1, 64, 16),
    ([1], [333], 8, 2, 64, 16),
    ([1, 1, 1, 1, 1], [1, 127, 128, 129, 1000], 8, 8, 128, 16),
    ([1, 1], [4100, 60], 32, 4, 128, 64),
    ([8, 8], [2048, 777], 16, 2, 128, 32),
    ([3, 0, 16, 1, 5], [100, 50, 16, 256, 511], 28, 4, 128, 32),          # a group of 7, a request with no window
    ([5, 9], [385, 129], 10, 2, 64, 128),                                 # a group of 5
    ([129, 33], [129, 200], 2, 2, 64, 16),
    ([300, 17, 64], [700, 17, 65], 8, 2, 128, 64),
    ([513], [1300], 1, 1, 128, 256),
    ([2, 70], [30, 90], 32, 1, 64, 16),                                   # one key head for all
]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("windows,lens,hq,hkv,d,page", SHAPES)
def test_windows_over_the_cache(ws, dtype, windows, lens, hq, hkv, d, page):
    run_and_check(Batch(windows, lens, hq, hkv, d, page, dtype, seed=sum(lens), pad_tokens=3), ws)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,page,heads_first", [(80, 16, False), (256, 16, True), (128, 7, False), (64, 1, False),
                                                (8, 16, True), (96, 4, False), (33, 5, True)])
def test_layouts_of_the_kernel_that_takes_every_layout(ws, dtype, d, page, heads_first):
    run_and_check(Batch([4, 1, 9], [130, 7, 30], 6, 2, d, page, dtype, seed=d, heads_first=heads_first), ws, heads_first)


def test_fp32_at_the_usual_sizes(ws):
    run_and_check(Batch([8, 1, 40], [333, 129, 40], 8, 2, 128, 16, F32), ws)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F32, 64)])
@pytest.mark.parametrize("window", [1, 16, 127, 128, 200])
def test_sliding_windows(ws, dtype, d, window):
    b = Batch([1, 8, 150, 3], [1000, 300, 420, 3], 8, 4, d, 16, dtype, seed=window)
    run_and_check(b, ws, window=window)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F32, 64)])
def test_rows_that_see_every_key(ws, dtype, d):
    b = Batch([8, 130, 1], [200, 130, 77], 8, 2, d, 32, dtype, seed=11)
    run_and_check(b, ws, full=True)
    run_and_check(b, ws, full=True, window=64)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F32, 64)])
def test_rows_that_see_nothing(ws, dtype, d):
    # windows longer than the cache (their first rows lie before it), a cache of length 0, no window at all
    run_and_check(Batch([5, 4, 0, 1, 200], [2, 0, 0, 5, 9], 4, 2, d, 16, dtype, seed=1), ws)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("scale", [0.0, -0.25, 3.0])
def test_scales(ws, dtype, d, scale):
    run_and_check(Batch([2, 9], [260, 40], 4, 2, d, 16, dtype, seed=8), ws, scale=scale)


@pytest.mark.parametrize("dtype,d,layout", [(BF16, 128, True), (F16, 64, False), (F32, 64, True)])
def test_heads_first_pages(ws, dtype, d, layout):
    run_and_check(Batch([6, 1, 20], [90, 300, 20], 8, 4, d, 32, dtype, seed=2, heads_first=layout), ws, layout)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F32, 64)])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
def test_what_a_row_does_not_see_has_no_influence(ws, dtype, d, poison):
    # the last two tokens of every window, and keys that slid out of the window, are poisoned in the cache; rows
    # that see none of them must be as if they were not there (Batch itself leaves NaN in every slot that is not cached)
    b = Batch([6, 4, 140], [300, 4, 300], 4, 2, d, 16, dtype, seed=21)
    clean = attend64(b, window=200)
    for r in range(b.n):
        for x in (b.k_pages, b.v_pages):
            for p in (b.lens[r] - 1, b.lens[r] - 2):
                x[b.table[r, p // b.page].item(), p % b.page] = poison
    r = 0
    for x in (b.k_pages, b.v_pages):
        for p in range(90):                                    # request 0's rows see keys 95.. and later
            x[b.table[r, p // b.page].item(), p % b.page] = poison
    q, kp, vp, table, qo, kv_len = b.gpu()
    got = sv.paged_attention(q, kp, vp, table, qo, kv_len, 140, window=200, ws=ws)
    rows = [t for r in range(b.n) for t in range(b.qo[r], b.qo[r + 1] - 2)]
    out, lse, tol, tol_l = (x[rows] for x in clean)
    diff = (got.out.double().cpu()[rows] - out).abs()
    assert (diff <= tol).all(), float((diff - tol).nan_to_num(1e9).max())
    assert ((got.lse.double().cpu()[rows] - lse).abs() <= tol_l).all()
    # the rows that see a NaN or +inf score give NaN
    if poison != -float("inf"):
        last = [b.qo[r + 1] - 1 for r in range(b.n)]
        assert got.out[last].isnan().any(-1).all()


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_an_infinite_value_stays_in_its_column(ws, dtype, d):
    b = Batch([3], [50], 2, 1, d, 16, dtype, seed=5)
    clean, _, tol, _ = attend64(b)
    b.v_pages[b.table[0, 48 // 16].item(), 48 % 16, 0, 5] = float("inf")     # the key of row 1
    q, kp, vp, table, qo, kv_len = b.gpu()
    got = sv.paged_attention(q, kp, vp, table, qo, kv_len, 3, ws=ws).out.double().cpu()
    assert ((got[0] - clean[0]).abs() <= tol[0]).all()
    assert (got[1:, :, 5] == math.inf).all()
    keep = [i for i in range(d) if i != 5]
    assert ((got[1:] - clean[1:]).abs()[..., keep] <= tol[1:][..., keep]).all()


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F32, 64)])
def test_scores_far_apart(ws, dtype, d):
    # maxima that grow by hundreds from key to key, in both directions
    b = Batch([1, 2, 30], [700, 300, 310], 4, 2, d, 16, dtype, seed=6, q_scale=12.0)
    for r in range(b.n):
        for p in range(b.lens[r]):
            at = b.table[r, p // b.page].item(), p % b.page
            b.k_pages[at] = (b.k_pages[at].float() * (0.02 * (p if r != 1 else b.lens[r] - p))).to(dtype)
    run_and_check(b, ws)


def test_refusals_on_the_device(ws):
    b = Batch([2, 2, 9, 2, 2], [40, 40, 40, 40, 40], 4, 2, 128, 16, BF16, seed=3)
    out, lse, tol, _ = attend64(b)
    q, kp, vp, table, qo, kv_len = b.gpu()
    table[0, 1] = b.n_pages
    table[1, 0] = -3
    kv_len[3] = 16 * table.shape[1] + 1
    status = torch.zeros(b.n, dtype=torch.int32, device="cuda")
    got = sv.paged_attention(q, kp, vp, table, qo, kv_len, 8, status=status, ws=ws)
    assert status.tolist() == [sv.ROW_BAD_LAYOUT] * 4 + [0]
    rows = slice(b.qo[4], b.qo[5])
    assert ((got.out.double().cpu() - out).abs()[rows] <= tol[rows]).all()
    kv_len[3] = -1
    status.zero_()
    sv.paged_attention(q, kp, vp, table, qo, kv_len, 9, status=status, ws=ws)
    assert status.tolist() == [sv.ROW_BAD_LAYOUT] * 2 + [0, sv.ROW_BAD_LAYOUT, 0]


def test_windows_outside_the_token_axis_are_refused(ws):
    b = Batch([2, 2], [40, 40], 4, 2, 128, 16, BF16, seed=3)
    q, kp, vp, table, qo, kv_len = b.gpu()
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    qo[2] = 100
    sv.paged_attention(q, kp, vp, table, qo, kv_len, 200, status=status, ws=ws)
    assert status.tolist() == [0, sv.ROW_BAD_LAYOUT]


def test_binding_refusals(ws):
    b = Batch([2, 2], [40, 40], 4, 2, 128, 16, BF16, seed=3)
    q, kp, vp, table, qo, kv_len = b.gpu()
    for bad in (dict(q=q.to(F16)), dict(q=q[..., :64]), dict(q=q.transpose(1, 2)), dict(table=table.long()),
                dict(table=table[:1]), dict(kv=kv_len.long()), dict(qo=qo[:2]), dict(vp=vp[:-1]), dict(q=q[:, :3])):
        a = dict(q=q, kp=kp, vp=vp, table=table, qo=qo, kv=kv_len)
        a.update(bad)
        with pytest.raises(sv.SVError):
            sv.paged_attention(a["q"], a["kp"], a["vp"], a["table"], a["qo"], a["kv"], 2, ws=ws)


def test_strided_queries_and_output(ws):
    b = Batch([8, 3], [150, 60], 4, 2, 128, 16, BF16, seed=14)
    out, _, tol, _ = attend64(b)
    q, kp, vp, table, qo, kv_len = b.gpu()
    packed = torch.zeros((b.tokens, 9, 128), dtype=BF16, device="cuda")
    packed[:, 1:5] = q
    dest = torch.zeros((b.tokens, 4, 136), dtype=BF16, device="cuda")[..., :128]
    got = sv.paged_attention(packed[:, 1:5], kp, vp, table, qo, kv_len, 8, out=dest, ws=ws)
    assert got.out is dest and ((dest.double().cpu() - out).abs() <= tol).all()
    # bases and strides off 16-byte boundaries
    flat = torch.zeros(b.tokens * 700 + 1, dtype=BF16, device="cuda")
    odd = torch.as_strided(flat, (b.tokens, 4, 128), (697, 131, 1), 1)
    odd.copy_(q)
    dest = torch.as_strided(torch.zeros_like(flat), (b.tokens, 4, 128), (697, 131, 1), 1)
    sv.paged_attention(odd, kp, vp, table, qo, kv_len, 8, out=dest, ws=ws)
    assert ((dest.double().cpu() - out).abs() <= tol).all()


def test_offsets_beyond_32_bits(ws):
    page, hkv, d = 64, 2, 128
    n_pages = 2 ** 31 // (page * hkv * d) + 40                  # over 2^31 elements a cache
    b = Batch([1, 4], [200, 130], 4, hkv, d, page, BF16, seed=17)
    out, lse, tol, tol_l = attend64(b)
    q, kp, vp, table, qo, kv_len = b.gpu()
    big = [torch.empty((n_pages, page, hkv, d), dtype=BF16, device="cuda") for _ in range(2)]
    shift = n_pages - b.n_pages
    for x, y in zip(big, (kp, vp)):
        x[shift:] = y
    got = sv.paged_attention(q, big[0], big[1], table + shift, qo, kv_len, 4, ws=ws)
    assert ((got.out.double().cpu() - out).abs() <= tol).all()
    assert ((got.lse.double().cpu() - lse).abs() <= tol_l).all()


def test_another_stream_repeats_and_a_graph(ws):
    b = Batch([1, 7, 2, 40], [3000, 900, 129, 640], 16, 2, 128, 32, BF16, seed=30)
    q, kp, vp, table, qo, kv_len = b.gpu()
    first = sv.paged_attention(q, kp, vp, table, qo, kv_len, 40, ws=ws)
    side, other = torch.cuda.Stream(), sv.Workspace("cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = [sv.paged_attention(q, kp, vp, table, qo, kv_len, 40, ws=other) for _ in range(3)]
    side.synchronize()
    for a in again:                                            # the same bits every time
        assert torch.equal(a.out, first.out) and torch.equal(a.lse, first.lse)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        captured = sv.paged_attention(q, kp, vp, table, qo, kv_len, 40, out=out, ws=ws)
    kv_len.sub_(torch.tensor([1, 5, 1, 7], dtype=torch.int32, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    want = sv.paged_attention(q, kp, vp, table, qo, kv_len, 40, ws=ws)
    assert torch.equal(out, want.out) and torch.equal(captured.lse, want.lse) and not torch.equal(out, first.out)


def test_a_result_does_not_depend_on_its_neighbours(ws):
    # the same request alone and in a batch: equal within the bound (its keys may be split elsewhere)
    b = Batch([4, 1, 60], [500, 1200, 300], 8, 2, 128, 16, BF16, seed=31)
    out, _, tol, _ = attend64(b)
    q, kp, vp, table, qo, kv_len = b.gpu()
    for r in range(b.n):
        rows = slice(b.qo[r], b.qo[r + 1])
        one = sv.paged_attention(q[rows], kp, vp, table[r:r + 1], torch.tensor([0, b.windows[r]], dtype=torch.int32,
                                 device="cuda"), kv_len[r:r + 1], b.windows[r], ws=ws)
        assert ((one.out.double().cpu() - out[rows]).abs() <= tol[rows]).all()
