"""What the beam and page calls refuse before any launch (no GPU), and their binding over stand-ins of tensors."""
import ctypes
import types

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.beam_cases import Pool, select64
from tests.test_attention_device import On, calls, workspace  # noqa: F401  (a fixture)

OK, BAD, WS, UNSUPPORTED = sv.SV_OK, sv.SV_ERR_INVALID_ARG, sv.SV_ERR_WORKSPACE, sv.SV_ERR_UNSUPPORTED
FAKE, ODD, NONE = 0x1000, 0x1001, None          # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    sv_build.build()
    return sv.load()


def select(lib, **change):
    a = dict(logits=FAKE, dt=0, s_item=400, s_beam=100, n=3, beams=4, vocab=100, scores=FAKE, finished=NONE, end=0, n_out=8,
             tokens=FAKE, parents=FAKE, out=FAKE, status=NONE, ws=FAKE, bytes=1 << 30, stream=NONE)
    a.update(change)
    return lib.sv_beam_select(*a.values())


def test_selection_refuses(lib):
    for change in (dict(logits=NONE), dict(scores=NONE), dict(tokens=NONE), dict(parents=NONE), dict(out=NONE), dict(n=-1),
                   dict(beams=0), dict(vocab=0), dict(n_out=0), dict(n_out=401), dict(dt=2), dict(dt=7), dict(logits=ODD),
                   dict(dt=1, logits=0x1002), dict(finished=FAKE, end=100), dict(finished=FAKE, end=-1)):
        assert select(lib, **change) == BAD, change
    for change in (dict(beams=129), dict(n_out=257), dict(vocab=524289), dict(n=1 << 21)):
        assert select(lib, **change) == UNSUPPORTED, change
    for change in (dict(ws=NONE), dict(ws=ODD), dict(bytes=100)):
        assert select(lib, **change) == WS, change
    assert select(lib, n=0, logits=NONE) == OK
    assert lib.sv_beam_workspace_size(3, 4, 100, 8) > 0
    for sizes in ((0, 4, 100, 8), (3, 129, 100, 8), (3, 4, 524289, 8), (3, 4, 100, 257), (3, 2, 4, 9)):
        assert lib.sv_beam_workspace_size(*sizes) == 0


def test_reordering_refuses(lib):
    def reorder(**change):
        a = dict(src=FAKE, si=64, sb=16, dst=0x9000, di=64, db=16, row=16, n=2, bi=4, bo=4, parents=FAKE, status=NONE, stream=NONE)
        a.update(change)
        return lib.sv_beam_reorder(*a.values())

    for change in (dict(src=NONE), dict(dst=NONE), dict(parents=NONE), dict(n=-1), dict(bi=0), dict(bo=0), dict(row=-1),
                   dict(dst=FAKE, bo=3), dict(dst=FAKE, di=128), dict(dst=FAKE, db=32)):
        assert reorder(**change) == BAD, change
    for change in (dict(n=65536), dict(bi=129), dict(bo=129), dict(row=(1 << 36) + 1)):
        assert reorder(**change) == UNSUPPORTED, change
    assert reorder(n=0) == OK and reorder(row=0) == OK


def test_forking_refuses(lib):
    def fork(ws=FAKE, size=1 << 34, parent=NONE, group=0, keep=FAKE, room=FAKE, copies=FAKE, **change):
        p = dict(table=FAKE, held=FAKE, ref=FAKE, ld=10, cols=10, n=4, pages=100, page=16)
        p.update(change)
        return lib.sv_kv_fork(sv.PagePool(*p.values()), parent, group, keep, room, copies, NONE, ws, size, NONE)

    for change in (dict(table=NONE), dict(held=NONE), dict(ref=NONE), dict(keep=NONE), dict(room=NONE), dict(copies=NONE),
                   dict(ld=9), dict(cols=-1), dict(n=-1), dict(pages=-1), dict(page=0), dict(group=-1)):
        assert fork(**change) == BAD, change
    for change in (dict(n=16385), dict(pages=(1 << 30) + 1), dict(n=16384, cols=16385, ld=16385)):
        assert fork(**change) == UNSUPPORTED, change
    for change in (dict(ws=NONE), dict(ws=ODD), dict(size=100)):
        assert fork(**change) == WS, change
    assert fork(n=0, table=NONE) == OK
    assert lib.sv_kv_fork_workspace_size(4, 10, 100) > 0 and lib.sv_kv_fork_workspace_size(16385, 10, 100) == 0


def test_copies_and_moves_refuse(lib):
    def cache(**change):
        c = dict(k=FAKE, v=FAKE, heads=2, v_heads=2, table=FAKE, ld=10, cols=10, pages=100, page=16)
        c.update(change)
        return sv.PagedKV(sv.Heads(c["k"], 128, 64, c["heads"]), sv.Heads(c["v"], 128, 64, c["v_heads"]), 2048, 2048, c["table"],
                          c["ld"], c["cols"], c["pages"], c["page"])

    def copy(dt=0, d=64, layers=1, copies=FAKE, m=3, **change):
        return lib.sv_kv_copy(cache(**change), dt, d, layers, 0, 0, copies, m, NONE, NONE)

    def compact(dt=0, d=64, layers=1, n=4, keep=FAKE, ld_keep=5, max_keep=5, n_keep=FAKE, **change):
        return lib.sv_kv_compact(cache(**change), dt, d, layers, 0, 0, n, NONE, keep, ld_keep, max_keep, n_keep, NONE, NONE)

    for call in (copy, compact):
        for change in (dict(k=NONE), dict(v=NONE), dict(k=ODD), dict(heads=0, v_heads=0), dict(v_heads=3), dict(page=0),
                       dict(pages=-1), dict(dt=3), dict(d=0), dict(layers=-1)):
            assert call(**change) == BAD, change
        for change in (dict(layers=32768), dict(d=1 << 19), dict(page=1 << 24, d=128)):
            assert call(**change) == UNSUPPORTED, change
        assert call(layers=0) == OK
    assert copy(copies=NONE) == BAD and copy(m=-1) == BAD and copy(m=0) == OK
    for change in (dict(n=-1), dict(max_keep=-1), dict(ld_keep=4), dict(keep=NONE), dict(n_keep=NONE), dict(table=NONE), dict(ld=9),
                   dict(cols=-1)):
        assert compact(**change) == BAD, change
    assert compact(n=65537) == UNSUPPORTED and compact(n=0) == OK
    assert compact(max_keep=(1 << 30) + 1, ld_keep=(1 << 30) + 1) == UNSUPPORTED


def test_host_tensors_are_refused():
    i = torch.zeros((2, 4), dtype=torch.int32)
    kv = torch.zeros((3, 16, 2, 64))
    with pytest.raises(sv.SVError, match="GPU"):
        sv.beam_select(torch.zeros((2, 4, 100)), torch.zeros((2, 4)), 4)
    with pytest.raises(sv.SVError, match="GPU"):
        sv.beam_reorder(torch.zeros((2, 4, 5)), i)
    with pytest.raises(sv.SVError, match="GPU"):
        sv.kv_fork(i, i[:, 0], i[0], 16, i[:, 0], i[:, 0])
    with pytest.raises(sv.SVError, match="GPU"):
        sv.kv_copy(kv, kv, torch.zeros((1, 3), dtype=torch.int32))
    with pytest.raises(sv.SVError, match="GPU"):
        sv.kv_compact(kv, kv, i, i, i[:, 0])


class Strided(On):
    """A stand-in that is not contiguous."""

    def __init__(self, device, shape, dtype, strides):
        super().__init__(device, shape, dtype)
        self.strides = strides

    def stride(self, d=None):
        return self.strides if d is None else self.strides[d]

    def is_contiguous(self):
        return False


def arguments(device):
    ints = lambda *shape: On(device, shape, torch.int32)                    # noqa: E731
    sized = lambda t, n: setattr(t, "element_size", lambda: n) or t         # noqa: E731
    return dict(logits=On(device, (3, 4, 100), torch.bfloat16), scores=On(device, (3, 4), torch.float32),
                finished=On(device, (3, 4), torch.bool), status=ints(3),
                out=sv.BeamOut(ints(3, 8), ints(3, 8), On(device, (3, 8), torch.float32)),
                state=sized(On(device, (3, 4, 7), torch.float32), 4), moved=sized(On(device, (3, 4, 7), torch.float32), 4),
                parents=ints(3, 4), table=ints(12, 9), held=ints(12), ref=ints(50), keep=ints(12), room=ints(12), parent=ints(12),
                copies=ints(12, 3), pages=On(device, (50, 16, 2, 64), torch.float16),
                layers=On(device, (5, 50, 16, 2, 64), torch.float16), kept=ints(12, 6), one=ints(1), of=ints(12))


CALLS = dict(
    sv_beam_select=lambda a, ws: sv.beam_select(a["logits"], a["scores"], 8, finished=a["finished"], out=a["out"],
                                                status=a["status"], ws=ws),
    sv_beam_reorder=lambda a, ws: sv.beam_reorder(a["state"], a["parents"], out=a["moved"], status=a["status"]),
    sv_kv_fork=lambda a, ws: sv.kv_fork(a["table"], a["held"], a["ref"], 16, a["keep"], a["room"], parent=a["parent"],
                                        group=4, copies=a["copies"], status=a["of"], ws=ws),
    sv_kv_copy=lambda a, ws: sv.kv_copy(a["layers"], a["layers"], a["copies"], status=a["one"]),
    sv_kv_compact=lambda a, ws: sv.kv_compact(a["pages"], a["pages"], a["table"], a["kept"], a["keep"], first=a["room"],
                                              status=a["of"]))
NEEDS = dict(sv_beam_select=("logits", "scores", "finished", "status"), sv_beam_reorder=("state", "moved", "parents", "status"),
             sv_kv_fork=("table", "held", "ref", "keep", "room", "parent", "copies", "of"),
             sv_kv_copy=("layers", "copies", "one"), sv_kv_compact=("pages", "table", "kept", "keep", "room", "of"))


@pytest.fixture
def made(calls, monkeypatch):                       # noqa: F811
    entry = lambda name: lambda *a: calls.append((name, torch.cuda.current_device())) or 0     # noqa: E731
    monkeypatch.setattr(sv, "_lib", types.SimpleNamespace(**{name: entry(name) for name in CALLS}))
    monkeypatch.setattr(sv, "beam_workspace_size", lambda *sizes: 1024)
    monkeypatch.setattr(sv, "kv_fork_workspace_size", lambda *sizes: 1024)
    return calls


@pytest.mark.parametrize("device", [0, 2])
def test_the_library_runs_on_the_tensors_device(made, device):
    for name, call in CALLS.items():
        call(arguments(device), workspace(device))
    assert made == [(name, device) for name in CALLS]
    assert torch.cuda.current_device() == 0


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_of_another_device_or_type_are_refused(made, name):
    for what in NEEDS[name]:
        if what in ("logits", "state", "layers", "pages"):
            continue                                # the tensor that says which device it is: the others are wrong then
        good = arguments(1)
        with pytest.raises(sv.SVError):
            CALLS[name](dict(good, **{what: arguments(0)[what]}), workspace(1))
        with pytest.raises(sv.SVError):
            CALLS[name](dict(good, **{what: On(1, good[what].shape, torch.float64)}), workspace(1))
        with pytest.raises(sv.SVError):
            CALLS[name](dict(good, **{what: On(1, (*good[what].shape, 2), good[what].dtype)}), workspace(1))
    assert made == []
    for what in ("sv_beam_select", "sv_kv_fork"):
        if name == what:
            with pytest.raises(sv.SVError, match="cuda:1"):
                CALLS[name](arguments(1), workspace(0))


def test_layouts_that_are_refused(made):
    a = arguments(0)
    f16 = torch.float16
    for logits in (On(0, (3, 4, 100), f16), On(0, (3, 400), torch.bfloat16),
                   Strided(0, (3, 4, 100), torch.bfloat16, (800, 200, 2))):
        with pytest.raises(sv.SVError):
            CALLS["sv_beam_select"](dict(a, logits=logits), workspace(0))
    for scores in (Strided(0, (3, 4), torch.float32, (8, 2)), On(0, (4, 3), torch.float32)):
        with pytest.raises(sv.SVError):
            CALLS["sv_beam_select"](dict(a, scores=scores), workspace(0))
    with pytest.raises(sv.SVError):
        sv.beam_select(a["logits"], a["scores"], 0, ws=workspace(0))
    for state in (On(0, (3,), f16), Strided(0, (3, 4, 7), torch.float32, (56, 14, 2))):
        state.element_size = lambda: 4
        with pytest.raises(sv.SVError):
            CALLS["sv_beam_reorder"](dict(a, state=state), workspace(0))
    for table in (Strided(0, (12, 9), torch.int32, (18, 2)), On(0, (11, 9), torch.int32)):
        with pytest.raises(sv.SVError):
            CALLS["sv_kv_fork"](dict(a, table=table), workspace(0))
        with pytest.raises(sv.SVError):
            CALLS["sv_kv_compact"](dict(a, table=table), workspace(0))
    for pages in (On(0, (50, 16, 128), f16), Strided(0, (50, 16, 2, 64), f16, (4096, 256, 128, 2))):
        with pytest.raises(sv.SVError):
            sv.kv_copy(pages, pages, a["copies"])
    with pytest.raises(sv.SVError):
        sv.kv_copy(a["pages"], a["layers"], a["copies"])
    assert made == []


def test_structures_match_the_header(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "sv.h"\nint main(void) {\n'
                   '  printf("%zu %zu %zu %d\\n", sizeof(sv_page_pool_t), offsetof(sv_page_pool_t, ref_count),\n'
                   "         offsetof(sv_page_pool_t, page_size), (int)SV_ROW_NO_PAGES);\n  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(sv.PagePool), sv.PagePool.ref_count.offset, sv.PagePool.page_size.offset, sv.ROW_NO_PAGES]


# the definitions that the device is held to, on cases worked out by hand
def test_the_definition_of_selection():
    log = lambda *p: torch.tensor(p).log()                       # noqa: E731
    logits = torch.stack([log(0.5, 0.25, 0.25) + 7, log(0.125, 0.75, 0.125) - 40])[None]
    scores = torch.tensor([[0.0, -0.1]])
    tokens, parents, s = select64(logits, scores, 4)
    assert tokens.tolist() == [[1, 0, 1, 2]] and parents.tolist() == [[1, 0, 0, 0]]
    want = torch.tensor([[0.75, 0.5, 0.25, 0.25]]).log().double() + torch.tensor([[-0.1, 0, 0, 0]])
    assert torch.allclose(s, want, atol=1e-6)
    tokens, parents, s = select64(logits, scores, 3, finished=torch.tensor([[False, True]]), end_token=2)
    assert tokens.tolist() == [[2, 0, 1]] and parents.tolist() == [[1, 0, 0]]
    tokens, parents, s = select64(torch.full((1, 2, 3), -float("inf")), scores, 6)
    assert tokens.tolist() == [[0, 1, 2, 0, 1, 2]] and (s == -float("inf")).all()


def test_the_definition_of_a_fork():
    pool = Pool(2, 3, 6, 4)
    pool.fork([0, 0], [6, 3])
    assert pool.table[0, :2].tolist() == [0, 1] and pool.table[1, 0] == 2 and pool.ref.tolist() == [1, 1, 1, 0, 0, 0]
    copies, _ = pool.fork([6, 6], [7, 9], [0, 0])                # the second of one parent: page 2 is free again
    assert copies.tolist() == [[-1, -1, -1], [1, 2, 2]]
    assert pool.table[1].tolist() == [0, 2, 3] and pool.ref.tolist() == [2, 1, 1, 1, 0, 0]
    copies, refused = pool.fork([0, 8], [0, 9])
    # request 1 gives its third page back and takes the lowest that is free, which request 0 gave back
    assert refused == [] and pool.ref.tolist() == [1, 1, 1, 0, 0, 0] and pool.held.tolist() == [0, 3]
    assert pool.table[1].tolist() == [0, 2, 1]
