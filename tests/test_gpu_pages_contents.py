"""What sv.kv_fork is for, without its rules: after every step each request reads the tokens that it should in the pages that it
holds, whatever the others write.  No number of a page is looked at but to read and write there."""
import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


@pytest.mark.parametrize("n,cols,n_pages,page,group", [(12, 9, 70, 4, 4), (12, 9, 30, 4, 0), (40, 12, 300, 7, 5), (9, 30, 270, 1, 3),
                                                       (1100, 6, 3000, 4, 10)])
def test_every_request_reads_its_own_tokens(n, cols, n_pages, page, group):
    g = torch.Generator().manual_seed(n + n_pages)
    rnd = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))      # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")          # noqa: E731
    table = ints([[0] * cols] * n)
    held, ref = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (n, n_pages))
    k = torch.full((n_pages, page, 1, 4), -1.0, device="cuda")                  # a token's key says which one it is
    v = torch.full((n_pages, page, 1, 4), -1.0, device="cuda")
    ws = sv.Workspace("cuda")
    text = [[] for _ in range(n)]                                               # the tokens that a request has
    fresh, served = 0, 0
    for s in range(14):
        low = [r // group * group if group else 0 for r in range(n)]
        size = [min(group, n - x) if group else n for x in low]
        parent = [rnd(0, size[r] - 1) if s % 3 else r - low[r] for r in range(n)]
        parent = [p if rnd(0, 2) else r - low[r] for r, p in enumerate(parent)]
        begun = [text[low[r] + parent[r]] for r in range(n)]
        keep = [len(t) if rnd(0, 3) else rnd(0, len(t)) for t in begun]
        room = [min(cols * page, x + (rnd(0, page + 2) if rnd(0, 3) else 0)) for x in keep]
        if s % 5 == 4:
            for r in range(0, n, 3):
                keep[r] = room[r] = 0
        status = torch.zeros(n, dtype=torch.int32, device="cuda")
        copies = sv.kv_fork(table, held, ref, page, ints(keep), ints(room), parent=ints(parent), group=group, status=status,
                            ws=ws)
        sv.kv_copy(k, v, copies)
        refused = status.tolist()
        assert set(refused) <= {0, sv.ROW_NO_PAGES}
        # everyone who has room appends, all at once; then all of it is read back
        text = [t[:x] for t, x in zip(begun, keep)]
        where, what = [], []
        rows, have = table.tolist(), held.tolist()
        for r in range(n):
            if refused[r]:
                assert have[r] == -(-keep[r] // page)
                continue
            assert have[r] == -(-room[r] // page)
            served += room[r] > keep[r]
            for p in range(keep[r], room[r]):
                where.append((rows[r][p // page], p % page))
                what.append(float(fresh))
                text[r] = text[r] + [fresh]
                fresh += 1
        assert len(set(where)) == len(where)                                    # no two write in one place
        if where:
            at = torch.tensor(where, device="cuda")
            k[at[:, 0], at[:, 1]] = torch.tensor(what, device="cuda")[:, None, None]
            v[at[:, 0], at[:, 1]] = -torch.tensor(what, device="cuda")[:, None, None]
        keys, values = k.cpu(), v.cpu()
        for r in range(n):
            if text[r]:
                p = torch.arange(len(text[r]))
                pages = torch.tensor(rows[r])[p // page]
                want = torch.tensor(text[r], dtype=torch.float32)
                assert torch.equal(keys[pages, p % page, 0, 0], want), (s, r)
                assert torch.equal(values[pages, p % page, 0, 3], -want), (s, r)
        # a count is that of the page's holders
        count = torch.zeros(n_pages, dtype=torch.int32)
        for r in range(n):
            for p in rows[r][:have[r]]:
                count[p] += 1
        assert torch.equal(ref.cpu(), count)
    assert served > 3 * n
