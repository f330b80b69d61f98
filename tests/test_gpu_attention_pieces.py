"""sv_paged_attention where its work is cut, joined and handed on: many short items, long ones over the whole GPU, items
that share tiles next to items that alternate, every page size and the cache layouts of serving runtimes."""
import math

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.attention_cases import Batch, attend64

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.fixture(scope="module")
def ws():
    return sv.Workspace("cuda")


def close(got, b, ref, rows=None):
    out, lse, tol, tol_l = ref
    sel = slice(0, b.qo[-1]) if rows is None else rows
    diff = (got.out.double().cpu() - out).abs()[sel]
    assert (diff <= tol[sel]).all(), float((diff - tol[sel]).nan_to_num(1e9).max())
    g, w = got.lse.double().cpu()[sel], lse[sel]
    seen = w != -math.inf
    assert torch.equal(g != -math.inf, seen) and ((g - w).abs()[seen] <= tol_l[sel][seen]).all()


def attend(b, ws, repeats=1, heads_first=False, **kw):
    """The result, with the status clear and the same bits every time."""
    q, kp, vp, table, qo, kv_len = b.gpu(heads_first)
    status = torch.zeros(b.n, dtype=torch.int32, device="cuda")
    first = None
    for _ in range(repeats):
        got = sv.paged_attention(q, kp, vp, table, qo, kv_len, max(b.windows), status=status, ws=ws, **kw)
        if first is None:
            first = got
        else:
            live = b.qo[-1]
            assert torch.equal(got.out[:live], first.out[:live]) and torch.equal(got.lse[:live], first.lse[:live])
    assert status.tolist() == [0] * b.n
    return first


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
def test_hundreds_of_short_requests(ws, dtype, d):
    g = torch.Generator().manual_seed(1)
    windows = torch.randint(1, 16, (256,), generator=g).tolist()
    lens = [max(w, n) for w, n in zip(windows, torch.randint(1, 700, (256,), generator=g).tolist())]
    b = Batch(windows, lens, 8, 2, d, 16, dtype, seed=2)
    close(attend(b, ws, repeats=150), b, attend64(b))


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("window", [0, 100])
def test_shared_and_alternating_tiles_side_by_side(ws, dtype, d, window):
    # groups of 2: windows of 64 tokens and less alternate tiles between the slots, larger ones share them
    windows = [1, 200, 3, 65, 64, 300, 1, 1, 129, 0, 70, 5, 257, 2]
    lens = [900, 200, 129, 300, 64, 1000, 2000, 1, 140, 77, 700, 5, 257, 1300]
    b = Batch(windows, lens, 4, 2, d, 32, dtype, seed=3)
    close(attend(b, ws, repeats=60, window=window), b, attend64(b, window=window))


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("windows,lens,hq,hkv", [([1], [40_000], 4, 1), ([8], [25_000], 8, 1), ([3, 1], [30_000, 7], 2, 2),
                                                 ([150], [9_000], 2, 1)])
def test_one_item_over_many_sms(ws, dtype, d, windows, lens, hq, hkv):
    b = Batch(windows, lens, hq, hkv, d, 64, dtype, seed=4)
    close(attend(b, ws, repeats=20), b, attend64(b))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 512])
@pytest.mark.parametrize("heads_first", [False, True])
def test_page_sizes(ws, d, page, heads_first):
    b = Batch([1, 9, 140], [700, 1100, 390], 4, 2, d, page, BF16, seed=page + d, heads_first=heads_first)
    close(attend(b, ws, heads_first=heads_first), b, attend64(b))


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 9, 12, 16, 32, 64])
def test_groups(ws, group):
    b = Batch([1, 11, 33], [300, 150, 260], 2 * group, 2, 128, 16, BF16, seed=group)
    close(attend(b, ws), b, attend64(b))


@pytest.mark.parametrize("d", [64, 128])
def test_keys_and_values_in_one_tensor(ws, d):
    b = Batch([2, 7, 90], [333, 128, 200], 6, 3, d, 16, BF16, seed=6)
    ref = attend64(b)
    q, kp, vp, table, qo, kv_len = b.gpu()
    for both in (torch.stack([kp, vp], dim=1), torch.stack([kp, vp], dim=3), torch.stack([kp, vp], dim=0)):
        at = both.shape.index(2)
        k, v = both.select(at, 0), both.select(at, 1)
        assert k.data_ptr() != v.data_ptr() and k.shape == kp.shape
        close(sv.paged_attention(q, k, v, table, qo, kv_len, 90, ws=ws), b, ref)


@pytest.mark.parametrize("d", [64, 128, 96])
def test_pages_that_nobody_sees_are_not_looked_at(ws, d):
    b = Batch([3, 1], [500, 400], 4, 2, d, 16, BF16, seed=7)
    ref = attend64(b, window=60)
    q, kp, vp, table, qo, kv_len = b.gpu()
    for r in range(2):
        gone = (b.lens[r] - b.windows[r] - 60 + 1) // 16       # pages wholly before the first row's window
        table[r, :gone] = -1
        table[r, -(-b.lens[r] // 16):] = 2 ** 30                # and those past the cache
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    close(sv.paged_attention(q, kp, vp, table, qo, kv_len, 3, window=60, ws=ws, status=status), b, ref)
    assert status.tolist() == [0, 0]


def test_a_wide_table_changes_nothing(ws):
    # short tables take one kernel, wide ones cut items between SMs and join them
    b = Batch([1, 4, 2], [500, 333, 129], 8, 2, 128, 16, BF16, seed=8)
    ref = attend64(b)
    q, kp, vp, table, qo, kv_len = b.gpu()
    assert table.shape[1] * 16 > 512
    close(sv.paged_attention(q, kp, vp, table[:, :32], qo, kv_len, 4, ws=ws), b, ref)
    wide = torch.full((3, 4000), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    close(sv.paged_attention(q, kp, vp, wide, qo, kv_len, 4, ws=ws), b, ref)


@pytest.mark.parametrize("d", [64, 128])
def test_other_requests_queries_do_not_matter(ws, d):
    b = Batch([2, 5, 3], [140, 260, 33], 8, 2, d, 16, BF16, seed=9)
    ref = attend64(b)
    for r in (0, 1, 2):
        keep = b.q.clone()
        for z in range(3):
            if z != r:
                b.q[b.qo[z]:b.qo[z + 1]] = float("nan")
        q, kp, vp, table, qo, kv_len = b.gpu()
        got = sv.paged_attention(q, kp, vp, table, qo, kv_len, 5, ws=ws)
        close(got, b, ref, rows=slice(b.qo[r], b.qo[r + 1]))
        b.q = keep


def test_a_workspace_full_of_anything(ws):
    # nothing in the workspace is read before it is written
    b = Batch([1, 3, 100], [5000, 800, 900], 8, 2, 128, 32, BF16, seed=10)
    ref = attend64(b)
    scratch = sv.Workspace("cuda")
    attend(b, scratch)
    for fill in (0, 255, 127):
        scratch.buf.fill_(fill)
        close(attend(b, scratch), b, ref)


def test_windows_of_a_whole_batch_without_tokens(ws):
    b = Batch([0, 0], [40, 0], 4, 2, 128, 16, BF16, pad_tokens=5)
    q, kp, vp, table, qo, kv_len = b.gpu()
    out = torch.full_like(q, 2.0)
    sv.paged_attention(q, kp, vp, table, qo, kv_len, 4, out=out, ws=ws)
    assert (out == 2.0).all()


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("windows,lens,window", [
    ([257, 1, 0, 128, 300, 129], [257, 40, 9, 513, 700, 131], 0),       # caches of up to 1,024 keys
    ([256, 129, 200, 3], [256, 200, 215, 0], 0),                        # of just over 256
    ([140, 256, 7], [140, 256, 7], 0),                                  # of no more than that
    ([500, 130, 1], [1100, 2000, 1500], 640),
    ([500, 130, 1], [1100, 2000, 1500], 641),
    ([400, 300], [1500, 300], 1),
    ([129, 260], [400, 2500], 130),
])
def test_prompts_with_a_key_head_for_every_query_head(ws, dtype, d, windows, lens, window):
    b = Batch(windows, lens, 2, 2, d, 16, dtype, seed=31)
    close(attend(b, ws, repeats=20, window=window), b, attend64(b, window=window))


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
def test_prompts_that_see_every_key_of_a_short_cache(ws, dtype, d):
    b = Batch([257, 130, 5], [600, 130, 700], 2, 2, d, 16, dtype, seed=32)
    close(attend(b, ws, repeats=5, full=True), b, attend64(b, full=True))
    close(attend(b, ws, repeats=5, full=True, window=200), b, attend64(b, full=True, window=200))


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
def test_poison_beyond_a_prompts_rows(ws, dtype, d):
    # a key that slid out of some rows' window and one that others do not see yet, in tiles that both slots read
    b = Batch([400, 300], [400, 1300], 2, 2, d, 16, dtype, seed=33)
    clean = attend64(b, window=150)
    spoiled = [(0, 200), (1, 1100)]
    for r, p in spoiled:
        b.v_pages[b.table[r, p // 16].item(), p % 16] = float("nan")
    q, kp, vp, table, qo, kv_len = b.gpu()
    got = sv.paged_attention(q, kp, vp, table, qo, kv_len, 400, window=150, ws=ws)
    out, _, tol, _ = clean
    diff = (got.out.double().cpu() - out).abs()
    for r, p in spoiled:
        first = b.lens[r] - b.windows[r]
        for i in range(b.windows[r]):
            row = b.qo[r] + i
            if first + i - 149 <= p <= first + i:
                assert got.out[row].isnan().all()
            else:
                assert (diff[row] <= tol[row]).all(), (r, i)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("others", [0, 40])
def test_a_prompt_of_more_items_than_a_warp_has_lanes(ws, dtype, d, others):
    b = Batch([2] * others + [4500, 3, 0], [70] * others + [4600, 900, 5], 2, 1, d, 64, dtype, seed=34)
    close(attend(b, ws, repeats=10, window=100), b, attend64(b, window=100))


@pytest.mark.parametrize("hq,hkv,d,page,dtype", [
    (5, 1, 256, 10, BF16), (6, 2, 80, 16, F16), (3, 3, 33, 7, torch.float32), (2, 2, 256, 64, torch.float32),
    (8, 1, 128, 24, BF16), (9, 3, 64, 16, torch.float32),
])
@pytest.mark.parametrize("windows,lens", [([1], [9000]), ([1, 3], [1, 4100]), ([2, 0, 1], [1030, 0, 130]),
                                          ([150, 90], [700, 90])])
def test_layouts_of_the_row_kernel(ws, hq, hkv, d, page, dtype, windows, lens):
    # heads that four rows do not divide, single rows; a CTA a unit of work, and clusters of them over long caches
    b = Batch(windows, lens, hq, hkv, d, page, dtype, seed=35)
    close(attend(b, ws, repeats=3), b, attend64(b))
    close(attend(b, ws, repeats=3, window=70), b, attend64(b, window=70))


def test_a_page_number_out_of_range_where_ctas_share_the_keys(ws):
    b = Batch([1, 2], [5000, 4000], 4, 1, 96, 16, BF16, seed=36)
    ref = attend64(b)
    q, kp, vp, table, qo, kv_len = b.gpu()
    table[0, 200] = b.n_pages
    table[0, 3] = -1
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    got = sv.paged_attention(q, kp, vp, table, qo, kv_len, 2, ws=ws, status=status)
    assert status.tolist() == [sv.ROW_BAD_LAYOUT, 0]
    close(got, b, ref, rows=slice(1, 3))
