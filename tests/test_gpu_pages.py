"""sv.kv_fork against the rules on the host, sv.kv_copy and sv.kv_compact against indexing."""
import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.beam_cases import Pool

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.fixture(scope="module")
def ws():
    return sv.Workspace("cuda")


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def step(pool, on, ws, keep, room, parent=None, group=0):
    """One fork step on both sides; the device's state has to be the host's."""
    table, held, ref = on
    status = torch.zeros(len(pool.held), dtype=torch.int32, device="cuda")
    copies = sv.kv_fork(table, held, ref, pool.page, ints(keep).cuda(), ints(room).cuda(),
                        parent=None if parent is None else ints(parent).cuda(), group=group, status=status, ws=ws)
    want, refused = pool.fork(keep, room, parent, group)
    assert torch.equal(held.cpu(), pool.held)
    assert torch.equal(copies.cpu(), want)
    assert torch.equal(ref.cpu(), pool.ref)
    assert torch.equal(table.cpu(), pool.table)
    assert status.tolist() == [sv.ROW_NO_PAGES if r in refused else 0 for r in range(len(pool.held))]
    return want, refused


# one CTA for all of it, and kernels for each step
SIZES = [(4, 6, 40, 4), (24, 40, 500, 16), (300, 20, 9000, 8), (40, 9000 // 16, 50000, 16), (7, 3000, 6000, 1)]


@pytest.mark.parametrize("n,max_pages,n_pages,page", SIZES)
@pytest.mark.parametrize("seed", [0, 1])
def test_steps_of_a_search(ws, n, max_pages, n_pages, page, seed):
    g = torch.Generator().manual_seed(seed * 100 + n)
    rnd = lambda lo, hi, m: torch.randint(lo, hi + 1, (m,), generator=g).tolist()      # noqa: E731
    pool = Pool(n, max_pages, n_pages, page, extra=(torch.rand(n_pages, generator=g) < 0.1).to(torch.int32))
    on = pool.gpu()
    lens = [min(x, max_pages * page) for x in rnd(0, max(1, n_pages * page // (2 * n)), n)]
    step(pool, on, ws, [0] * n, lens)
    for s in range(8):
        parent = rnd(0, n - 1, n) if s % 2 else [r if x < n // 2 else x for r, x in enumerate(rnd(0, n - 1, n))]
        have = [int(h) * page for h in pool.held]
        keep = [min(lens[p], have[p]) for p in parent]
        keep = [max(0, k - d) if s % 3 == 2 else k for k, d in zip(keep, rnd(0, 2 * page, n))]
        lens = [min(max_pages * page, k + d) for k, d in zip(keep, rnd(0, page + 1, n))]
        if s == 5:
            lens[0], keep[0] = 0, 0                        # one is done
        step(pool, on, ws, keep, lens, parent)
        lens = [min(x, int(h) * page) for x, h in zip(lens, pool.held)]
    step(pool, on, ws, [0] * n, [0] * n)                   # everything goes back
    assert int(pool.held.sum()) == 0 and int(pool.ref.max()) <= 1


@pytest.mark.parametrize("beams", [1, 3, 8])
def test_groups_and_no_parents(ws, beams):
    n, page = 6 * beams, 16
    pool = Pool(n, 30, 2000, page)
    on = pool.gpu()
    g = torch.Generator().manual_seed(beams)
    lens = [int(x) for x in torch.randint(1, 300, (n,), generator=g)]
    step(pool, on, ws, [0] * n, lens)
    for s in range(5):
        parent = torch.randint(0, beams, (n,), generator=g).tolist()
        keep = [lens[r // beams * beams + p] for r, p in enumerate(parent)]
        lens = [k + 1 + s for k in keep]
        step(pool, on, ws, keep, lens, parent, group=beams)
        keep = [max(0, x - 5) for x in lens]               # rejected tokens go back, room for a window
        lens = [k + 9 for k in keep]
        step(pool, on, ws, keep, lens)


def test_who_writes_on_a_shared_page(ws):
    page = 8
    # two beams of one parent: the first stays, the second copies
    pool = Pool(3, 4, 20, page)
    on = pool.gpu()
    step(pool, on, ws, [0, 0, 0], [11, 5, 3])
    want, _ = step(pool, on, ws, [11, 11, 3], [12, 12, 3], [0, 0, 2])
    assert want[0].tolist() == [-1, -1, -1] and want[1, 2] == 3 and want[2].tolist() == [-1, -1, -1]
    # one who only reads stands by: every writer copies
    pool = Pool(3, 4, 20, page)
    on = pool.gpu()
    step(pool, on, ws, [0, 0, 0], [11, 0, 0])
    want, _ = step(pool, on, ws, [11, 11, 11], [12, 11, 12], [0, 0, 0])
    assert want[:, 2].tolist() == [3, -1, 3]
    # a holder outside the table counts too
    pool = Pool(2, 4, 20, page)
    pool.ref[1] += 1
    on = pool.gpu()
    step(pool, on, ws, [0, 0], [6, 0])                     # page 0, which nobody else has
    want, _ = step(pool, on, ws, [6, 0], [7, 0])
    assert want[0].tolist() == [-1, -1, -1]
    pool.ref[0] += 1
    on[2].copy_(pool.ref)
    want, _ = step(pool, on, ws, [7, 0], [8, 0])
    assert want[0].tolist() == [0, 2, 7]
    # shorter beginnings of one page: the longest stays, whoever is refused keeps what it reads
    pool = Pool(3, 2, 3, page)
    on = pool.gpu()
    step(pool, on, ws, [0, 0, 0], [7, 0, 0])
    want, refused = step(pool, on, ws, [3, 7, 5], [4, 8, 16], [0, 0, 0])
    assert want[0].tolist() == [0, 1, 3] and want[1].tolist() == [-1, -1, -1] and refused == [2]
    assert pool.ref.tolist() == [2, 1, 0] and pool.held.tolist() == [1, 1, 1]


def test_an_empty_pool_and_whole_pages(ws):
    pool = Pool(5, 4, 4, 2)
    on = pool.gpu()
    _, refused = step(pool, on, ws, [0] * 5, [3, 3, 2, 1, 0])
    assert refused == [2, 3]                               # their places in the line lie past the free pages
    _, refused = step(pool, on, ws, [2, 3, 0, 0, 0], [2, 3, 2, 2, 0])
    assert refused == [3]
    step(pool, on, ws, [0] * 5, [0] * 5)
    assert pool.ref.tolist() == [0] * 4


@pytest.mark.parametrize("n,max_pages,n_pages", [(6, 8, 100), (6, 8, 60000)])
def test_what_is_refused_is_refused_by_request(ws, n, max_pages, n_pages):
    page = 16
    pool = Pool(n, max_pages, n_pages, page)
    on = pool.gpu()
    step(pool, on, ws, [0] * n, [40, 50, 60, 70, 80, 90])
    before = [t.clone() for t in on]
    bad = sv.ROW_BAD_LAYOUT
    for r, keep, room, parent in ((1, -1, 40, 1), (2, 65, 70, 2), (3, 50, 49, 3), (4, 80, 129, 4), (5, 1, 1, -1), (0, 1, 1, 6),
                                  (1, 81, 90, 0)):
        keeps, rooms = [40, 50, 60, 70, 80, 90], [40, 50, 60, 70, 80, 90]
        parents = list(range(n))
        keeps[r], rooms[r], parents[r] = keep, room, parent
        status = torch.zeros(n, dtype=torch.int32, device="cuda")
        copies = sv.kv_fork(*on, page, ints(keeps).cuda(), ints(rooms).cuda(), parent=ints(parents).cuda(), status=status,
                            ws=ws)
        assert status.tolist() == [bad if i == r else 0 for i in range(n)]
        assert (copies == -1).all()
        for a, b in zip(before, on):
            assert torch.equal(a, b)
    # a parent outside its group
    status.zero_()
    sv.kv_fork(*on, page, ints([40, 50, 60, 70, 80, 90]).cuda(), ints([40, 50, 60, 70, 80, 90]).cuda(),
               parent=ints([0, 1, 2, 0, 1, 2]).cuda(), group=3, status=status, ws=ws)
    assert status.tolist() == [0] * 6
    status.zero_()
    sv.kv_fork(*on, page, ints([40] * 6).cuda(), ints([40] * 6).cuda(), parent=ints([0, 1, 3, 0, 1, 2]).cuda(), group=3,
               status=status, ws=ws)
    assert status.tolist() == [0, 0, bad, 0, 0, 0]


def test_broken_tables_and_counts_are_not_followed(ws):
    pool = Pool(4, 6, 50, 16)
    on = pool.gpu()
    step(pool, on, ws, [0] * 4, [40, 50, 60, 70])
    table, held, ref = on
    table[1, 1], table[2, 0] = 50, -3
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    sv.kv_fork(table, held, ref, 16, ints([40, 0, 60, 70]).cuda(), ints([41, 0, 60, 70]).cuda(), status=status, ws=ws)
    assert status.tolist() == [0, sv.ROW_BAD_LAYOUT, 0, 0]         # request 2 keeps its page as it is
    assert held.tolist() == [3, 0, 4, 5]
    held[3] = 7
    status.zero_()
    sv.kv_fork(table, held, ref, 16, ints([40, 0, 60, 70]).cuda(), ints([40, 0, 60, 70]).cuda(), status=status, ws=ws)
    assert status.tolist() == [0, 0, 0, sv.ROW_BAD_LAYOUT] and held.tolist() == [3, 0, 4, 7]
    held[3] = 5
    status.zero_()
    before = ref.clone()
    sv.kv_fork(table, held, ref, 16, ints([60, 0, 60, 70]).cuda(), ints([60, 0, 60, 70]).cuda(), parent=ints([2, 1, 2, 3]).cuda(),
               status=status, ws=ws)
    assert status.tolist() == [sv.ROW_BAD_LAYOUT, 0, 0, 0]         # takes -3 with the rest
    assert table[0, :4].tolist() == table[2, :4].tolist()
    assert int(ref.sum()) == int(before.sum())                     # three pages given back, three that count taken


@pytest.mark.parametrize("large", [False, True])
def test_forks_are_captured_and_streams_are_the_callers(large):
    n, page = (12, 16) if not large else (600, 16)
    n_pages = 4000 if not large else 60000
    pool, ws = Pool(n, 40, n_pages, page), sv.Workspace("cuda")
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


# ---------------------------------------------------------------------------------------------------------------
# Copies
# ---------------------------------------------------------------------------------------------------------------
def cache_of(layers, n_pages, page, heads, d, dtype, order, seed=0):
    """K and V pages on the device in one of several orders; layers 0: no axis of layers."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lead = (layers,) if layers else ()
    make = lambda *dims: torch.randn(lead + dims, generator=g, device="cuda").to(dtype)      # noqa: E731
    if order == "tokens":
        return make(n_pages, page, heads, d), make(n_pages, page, heads, d)
    if order == "heads":
        return make(n_pages, heads, page, d).transpose(-3, -2), make(n_pages, heads, page, d).transpose(-3, -2)
    if order == "both":                                    # keys and values side by side
        kv = make(n_pages, 2, page, heads, d)
        return kv.select(-4, 0), kv.select(-4, 1)
    odd = make(n_pages, page, heads, d + 3)                # heads that begin anywhere, values the other way round
    return odd[..., 1:d + 1], make(n_pages, heads, page, d).transpose(-3, -2)


LAYOUTS = ["tokens", "heads", "both", "odd"]


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F32, 64), (BF16, 80), (BF16, 20), (F16, 7), (F32, 1)])
@pytest.mark.parametrize("order", LAYOUTS)
@pytest.mark.parametrize("layers", [0, 1, 3])
def test_pages_are_copied(dtype, d, order, layers):
    n_pages, page, heads = 30, 16, 3
    k, v = cache_of(layers, n_pages, page, heads, d, dtype, order)
    g = torch.Generator().manual_seed(d)
    where = torch.randperm(n_pages, generator=g)
    copies = torch.stack([where[:10], where[10:20], torch.tensor([1, 16, 0, 5, 15, 16, 2, 3, 9, 7])], 1).to(torch.int32)
    copies[3, 0] = -1
    copies[4, 1] = -1
    want = [k.clone(), v.clone()]
    for t in want:
        for i, (src, dst, m) in enumerate(copies.tolist()):
            if i not in (3, 4):
                t[..., dst, :m, :, :] = t[..., src, :m, :, :]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.kv_copy(k, v, copies.cuda(), status=status)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and int(status) == 0


@pytest.mark.parametrize("page,heads,d", [(1, 1, 8), (128, 8, 128), (7, 5, 96), (1024, 2, 256)])
def test_pages_of_other_sizes(page, heads, d):
    k, v = cache_of(2, 9, page, heads, d, BF16, "tokens")
    copies = ints([[0, 5, page], [1, 6, max(1, page // 2)], [0, 7, page - page // 3]]).cuda()    # one page to several
    want = [k.clone(), v.clone()]
    for t in want:
        for src, dst, m in copies.tolist():
            t[:, dst, :m] = t[:, src, :m]
    sv.kv_copy(k, v, copies)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_bad_copies_are_left_out():
    k, v = cache_of(0, 6, 8, 2, 64, BF16, "tokens")
    before = k.clone(), v.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in ([6, 1, 3], [1, 6, 3], [0, 1, 9], [0, 1, -2], [2 ** 31 - 1, 0, 1]):
        status.zero_()
        sv.kv_copy(k, v, ints([bad, [-1, -1, -1]]).cuda(), status=status)
        sv.kv_copy(k, v, ints([bad]).cuda())
        assert int(status) == sv.ROW_BAD_LAYOUT
        assert torch.equal(k, before[0]) and torch.equal(v, before[1])
    sv.kv_copy(k, v, torch.zeros((0, 3), dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------------------------------------------------------
# Tokens that move together
# ---------------------------------------------------------------------------------------------------------------
def compacted(t, table, first, keep, n_keep, page):
    """The pages `t` after the move, by sequences on the host's side of things."""
    out = t.clone()
    for r, n in enumerate(n_keep):
        src = [first[r] + keep[r][j] for j in range(n)]
        for j, p in enumerate(src):
            q = first[r] + j
            out[..., table[r][q // page], q % page, :, :] = t[..., table[r][p // page], p % page, :, :]
    return out


def compact_case(n, page, window, seed, share=0.5, first_hi=50):
    g = torch.Generator().manual_seed(seed)
    first = torch.randint(0, first_hi + 1, (n,), generator=g).tolist()
    cols = -(-(max(first) + window) // page)
    table = torch.randperm(n * cols + 2, generator=g)[: n * cols].view(n, cols).tolist()
    keep, n_keep = [], []
    for r in range(n):
        row = [i for i in range(window) if float(torch.rand((), generator=g)) < share]
        n_keep.append(len(row))
        keep.append(row + [-5] * (window - len(row)))
    return first, table, keep, n_keep, n * cols + 2


def run_compact(k, v, first, table, keep, n_keep, page):
    want = [compacted(t, table, first, keep, n_keep, page) for t in (k, v)]
    status = torch.zeros(len(first), dtype=torch.int32, device="cuda")
    sv.kv_compact(k, v, ints(table).cuda(), ints(keep).cuda(), ints(n_keep).cuda(), first=ints(first).cuda(), status=status)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert status.tolist() == [0] * len(first)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F32, 64), (BF16, 20), (F16, 7)])
@pytest.mark.parametrize("order", LAYOUTS)
@pytest.mark.parametrize("layers", [0, 2])
def test_kept_tokens_move_together(dtype, d, order, layers):
    first, table, keep, n_keep, n_pages = compact_case(5, 16, 37, d)
    k, v = cache_of(layers, n_pages, 16, 3, d, dtype, order)
    run_compact(k, v, first, table, keep, n_keep, 16)


@pytest.mark.parametrize("n,window,share", [(1, 1, 1.0), (3, 8, 0.0), (2, 64, 1.0), (2, 600, 0.9), (1, 3000, 0.5), (40, 63, 0.1),
                                            (3, 2500, 0.01)])
@pytest.mark.parametrize("page,heads", [(16, 8), (5, 1), (64, 2)])
def test_windows_of_all_lengths(n, window, share, page, heads):
    first, table, keep, n_keep, n_pages = compact_case(n, page, window, window, share)
    k, v = cache_of(0, n_pages, page, heads, 64, BF16, "tokens")
    run_compact(k, v, first, table, keep, n_keep, page)


@pytest.mark.parametrize("layers,n,window,share", [(40, 6, 30, 0.4), (33, 64, 20, 0.3), (3, 300, 70, 0.5), (5, 1, 5000, 0.7)])
def test_many_layers_and_long_lists(layers, n, window, share):
    first, table, keep, n_keep, n_pages = compact_case(n, 16, window, layers, share)
    keep = [row[:max(n_keep)] for row in keep]                # a short list, whatever the window
    k, v = cache_of(layers, n_pages, 16, 2, 64, F16, "tokens")
    v = torch.cat([v, v], -1)[..., 17:81]                     # values in other places than the keys
    run_compact(k, v, first, table, keep, n_keep, 16)


def test_every_second_token_and_no_first():
    # overlapping moves of a page at a time, from the first token of the cache
    page, n_keep = 16, 500
    k, v = cache_of(0, 70, page, 2, 128, BF16, "heads")
    table, keep = [list(range(69, 0, -1))], [[2 * j + 1 for j in range(n_keep)]]
    want = [compacted(t, table, [0], keep, [n_keep], page) for t in (k, v)]
    sv.kv_compact(k, v, ints(table).cuda(), ints(keep).cuda(), ints([n_keep]).cuda())
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_bad_lists_are_their_requests_business():
    page = 16
    first, table, keep, n_keep, n_pages = compact_case(8, page, 40, 3, 0.5, 20)
    n_keep = [max(n, 6) for n in n_keep]
    keep = [list(range(1, 41)) for _ in range(8)]
    k, v = cache_of(0, n_pages, page, 2, 64, BF16, "tokens")
    good = [r for r in range(8) if r in (0, 7)]
    want = [compacted(t, table, first, keep, [n if r in good else 0 for r, n in enumerate(n_keep)], page) for t in (k, v)]
    broken_t, broken_k, broken_f, broken_n = [r[:] for r in table], [r[:] for r in keep], first[:], n_keep[:]
    broken_n[1] = -1
    broken_n[2] = 41
    broken_f[3] = -1
    broken_k[4][2] = 2                                     # not ascending
    broken_k[5][5] = 2 ** 31 - 1                           # past the table
    broken_t[6] = [n_pages] * len(table[6])
    status = torch.zeros(8, dtype=torch.int32, device="cuda")
    sv.kv_compact(k, v, ints(broken_t).cuda(), ints(broken_k).cuda(), ints(broken_n).cuda(), first=ints(broken_f).cuda(),
                  status=status)
    assert status.tolist() == [0] + [sv.ROW_BAD_LAYOUT] * 6 + [0]
    mine = sorted(p for r in good for p in table[r])
    assert torch.equal(k[mine], want[0][mine]) and torch.equal(v[mine], want[1][mine])
    others = sorted(set(range(n_pages)) - {p for r in (0, 4, 5, 7) for p in table[r]})
    assert torch.equal(k[others], want[0][others])         # and nothing else


def test_a_long_cache_has_offsets_past_32_bits():
    # 2.1e9 elements a tensor: the last pages' bytes lie past 2^32
    page, heads, d, n_pages = 64, 8, 128, 33000
    k = torch.zeros((n_pages, page, heads, d), dtype=BF16, device="cuda")
    last = n_pages - 1
    k[last - 1] = 1.0
    k[last, 5] = 3.0
    sv.kv_copy(k, k, ints([[last - 1, last, 4]]).cuda())
    assert (k[last, :4] == 1).all() and (k[last, 5] == 3).all() and (k[last, 4] == 0).all()
    sv.kv_compact(k, k, ints([[last, 0]]).cuda(), ints([[5]]).cuda(), ints([1]).cuda())
    assert (k[last, 0] == 3).all() and (k[last, 1] == 1).all()


@pytest.mark.parametrize("layers", [0, 2])
def test_one_tensor_for_keys_and_values(layers):
    # moved once: twice would take the second time what the first has put there
    page, n_keep = 16, 900
    k, _ = cache_of(layers, 130, page, 2, 64, BF16, "tokens")
    table, keep = [list(range(120, 0, -1))], [[2 * j + 1 for j in range(n_keep)]]
    want = compacted(k, table, [0], keep, [n_keep], page)
    sv.kv_compact(k, k, ints(table).cuda(), ints(keep).cuda(), ints([n_keep]).cuda())
    assert torch.equal(k, want)
    want[..., 125, :9, :, :] = want[..., 3, :9, :, :]
    sv.kv_copy(k, k, ints([[3, 125, 9]]).cuda())
    assert torch.equal(k, want)
