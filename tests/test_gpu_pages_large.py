"""sv.kv_fork in both of its forms: one cluster, and a kernel for each step where rows or pages are many.

The form is read off the call itself: the kernels of a captured one."""
import ctypes

import pytest
import torch

import tests.test_gpu_pages as small
from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.beam_cases import Pool

pytestmark = pytest.mark.gpu

ints, step = small.ints, small.step


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.fixture(scope="module")
def ws():
    return sv.Workspace("cuda")


def kernels_of(n, max_pages, n_pages, page, ws):
    """How many kernels a call of these sizes is."""
    table = torch.zeros((n, max_pages), dtype=torch.int32, device="cuda")
    held, ref, zero = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (n, n_pages, n))
    copies = torch.empty((n, 3), dtype=torch.int32, device="cuda")
    call = lambda: sv.kv_fork(table, held, ref, page, zero, zero, copies=copies, ws=ws)      # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    nodes = ctypes.c_size_t()
    get = ctypes.CDLL("libcuda.so.1").cuGraphGetNodes
    get.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)]
    assert get(graph.raw_cuda_graph(), None, ctypes.byref(nodes)) == 0
    return nodes.value


# 1,024 tiles of 256 columns, and 64 of 4,096 pages: the last sizes of one cluster, and the first past them
FORMS = [(1024, 20, 9000, 8, 1), (1025, 20, 9000, 8, 3), (1100, 20, 33000, 8, 3), (102, 2560, 40000, 4, 1),
         (113, 2305, 40000, 4, 3), (6, 40, 262144, 16, 1), (6, 40, 262145, 16, 3)]


@pytest.mark.parametrize("n,max_pages,n_pages,page,kernels", FORMS)
def test_steps_of_a_search_in_both_forms(ws, n, max_pages, n_pages, page, kernels):
    assert kernels_of(n, max_pages, n_pages, page, ws) == kernels
    small.test_steps_of_a_search(ws, n, max_pages, n_pages, page, 2)


@pytest.mark.parametrize("n,kernels", [(900, 1), (1100, 3), (2300, 3)])
def test_a_pool_that_runs_out(ws, n, kernels):
    page, n_pages = 8, 3 * n
    assert kernels_of(n, 12, n_pages, page, ws) == kernels
    pool = Pool(n, 12, n_pages, page)
    on = pool.gpu()
    g = torch.Generator().manual_seed(n)
    rnd = lambda hi: torch.randint(0, hi + 1, (n,), generator=g).tolist()      # noqa: E731
    lens = rnd(6 * page)
    _, refused = step(pool, on, ws, [0] * n, lens)
    many = [len(refused)]
    for s in range(4):
        have = (pool.held * page).tolist()
        parent = [p if r % 2 else r for r, p in enumerate(rnd(n - 1))]
        keep = [min(lens[p], have[p]) // (1 if r % 5 else 2) for r, p in enumerate(parent)]
        lens = [min(12 * page, k + d) for k, d in zip(keep, rnd(2 * page))]
        _, refused = step(pool, on, ws, keep, lens, parent)
        lens = [keep[r] if r in refused else x for r, x in enumerate(lens)]
        many.append(len(refused))
    assert max(many) > 0 and min(many) < n // 2
    step(pool, on, ws, [0] * n, [0] * n)
    assert int(pool.ref.max()) == 0


def test_what_is_refused_is_refused_by_request_in_three_kernels(ws):
    assert kernels_of(6, 8, 300000, 16, ws) == 3
    small.test_what_is_refused_is_refused_by_request(ws, 6, 8, 300000)


def test_broken_tables_are_not_followed_in_three_kernels(ws):
    n, page = 1030, 16
    assert kernels_of(n, 6, 9000, page, ws) == 3
    pool = Pool(n, 6, 9000, page)
    on = pool.gpu()
    lens = [40 + r % 50 for r in range(n)]
    step(pool, on, ws, [0] * n, lens)
    table, held, ref = on
    table[1, 1], table[1029, 0] = 9000, -3
    before = ref.clone()
    keep, room, parent = lens[:], lens[:], list(range(n))
    keep[1] = room[1] = 0                           # gives 9000 back
    keep[7] = room[7] = 33
    parent[7] = 1029                                # takes -3 with the rest
    status = torch.zeros(n, dtype=torch.int32, device="cuda")
    copies = sv.kv_fork(table, held, ref, page, ints(keep).cuda(), ints(room).cuda(), parent=ints(parent).cuda(),
                        status=status, ws=ws)
    want = [0] * n
    want[1] = want[7] = sv.ROW_BAD_LAYOUT
    assert status.tolist() == want and (copies == -1).all()
    assert held[1] == 0 and held[7] == 3 and torch.equal(table[7, :3], table[1029, :3])
    # request 1 gives two pages back that count, 7 its own three for two that count
    assert int(ref.sum()) == int(before.sum()) - 2 - 3 + 2


def test_three_kernels_are_captured():
    n, page, n_pages = 1100, 16, 60000
    pool, ws = Pool(n, 40, n_pages, page), sv.Workspace("cuda")
    assert kernels_of(n, 40, n_pages, page, ws) == 3
    on = pool.gpu()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(pool, on, ws, [0] * n, [100] * n)
    torch.cuda.current_stream().wait_stream(side)
    keep, room = ints([100] * n).cuda(), ints([101] * n).cuda()
    parent, copies = ints([0] * n).cuda(), torch.empty((n, 3), dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sv.kv_fork(*on, page, keep, room, parent=parent, copies=copies, ws=ws)
    length = 100
    for s in range(4):
        parents = [(r * 7 + s) % n if r % 3 else r for r in range(n)]
        keep.fill_(length)
        room.fill_(length + 5)
        parent.copy_(ints(parents))
        graph.replay()
        want, _ = pool.fork([length] * n, [length + 5] * n, parents)
        length += 5
        for a, b in zip(on + (copies,), (pool.table, pool.held, pool.ref, want)):
            assert torch.equal(a.cpu(), b)


def test_as_many_requests_as_there_may_be(ws):
    n, page = 16384, 4
    pool = Pool(n, 3, 40000, page)
    on = pool.gpu()
    g = torch.Generator().manual_seed(1)
    rnd = lambda hi: torch.randint(0, hi + 1, (n,), generator=g).tolist()      # noqa: E731
    lens = rnd(5)
    step(pool, on, ws, [0] * n, lens)
    parent = rnd(n - 1)
    keep = [lens[p] for p in parent]
    step(pool, on, ws, keep, [k + 1 for k in keep], parent)
    keep = [max(0, k - 1) for k in keep]
    step(pool, on, ws, keep, [k + 4 for k in keep])


def test_a_pool_of_more_tiles_than_a_block_counts_at_once(ws):
    # 1,050 tiles of pages; what is free lies in few of them, most of it in the last ones
    n, page, n_pages = 5, 16, 4_300_000
    extra = torch.ones(n_pages, dtype=torch.int32)
    extra[3::50_000] = 0
    extra[4_290_000:] = 0
    pool = Pool(n, 100, n_pages, page, extra=extra)
    on = pool.gpu()
    step(pool, on, ws, [0] * n, [1600, 3, 800, 0, 33])
    step(pool, on, ws, [1600, 1590, 3, 15, 3], [1600, 1600, 50, 40, 4], [0, 0, 1, 2, 1])
    step(pool, on, ws, [0] * n, [0] * n)
    assert torch.equal(pool.ref, extra)
