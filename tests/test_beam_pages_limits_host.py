"""Numbers that the library takes in 32 bits are refused where they need more, not cut down to something else."""
import pytest
import torch

from speculative_decoding_verification_rows_gb300 import sv
from tests.test_attention_device import On, calls, workspace      # noqa: F401  (a fixture)
from tests.test_beam_pages_host import CALLS, Strided, arguments, made      # noqa: F401  (a fixture)

BIG = 2 ** 32 + 5                                   # 5 in 32 bits
INT, F32, BF16 = torch.int32, torch.float32, torch.bfloat16


def refused(name, **change):
    with pytest.raises(sv.SVError):
        CALLS[name](dict(arguments(0), **change), workspace(0))


def test_sizes_past_32_bits(made, monkeypatch):     # noqa: F811
    monkeypatch.undo()                              # the workspace sizes are the library's own
    sv.load(build_if_missing=True)
    for size, sizes in ((sv.beam_workspace_size, (3, 4, 100, 8)), (sv.kv_fork_workspace_size, (12, 9, 50))):
        assert size(*sizes) > 0
        for i in range(len(sizes)):
            with pytest.raises(sv.SVError):
                size(*sizes[:i], sizes[i] + 2 ** 32, *sizes[i + 1:])


def test_selection(made):                           # noqa: F811
    a = arguments(0)
    select = lambda end: sv.beam_select(a["logits"], a["scores"], 8, finished=a["finished"], end_token=end, out=a["out"],   # noqa: E731
                                        ws=workspace(0))
    for end in (BIG, -1, 100, -2 ** 32 + 5):
        with pytest.raises(sv.SVError):
            select(end)
    assert made == []
    select(99)
    sv.beam_select(a["logits"], a["scores"], 8, end_token=-1, out=a["out"], ws=workspace(0))     # of no beam
    assert len(made) == 2


def test_reordering(made):                          # noqa: F811
    sized = lambda shape: setattr(t := On(0, shape, F32), "element_size", lambda: 4) or t        # noqa: E731
    refused("sv_beam_reorder", state=sized((BIG, 4, 7)), moved=sized((BIG, 4, 7)), parents=On(0, (BIG, 4), INT),
            status=On(0, (BIG,), INT))
    refused("sv_beam_reorder", state=sized((3, BIG, 7)))
    refused("sv_beam_reorder", moved=sized((3, BIG, 7)), parents=On(0, (3, BIG), INT))
    assert made == []


def test_pages(made):                               # noqa: F811
    a = arguments(0)
    fork = lambda page, group: sv.kv_fork(a["table"], a["held"], a["ref"], page, a["keep"], a["room"], parent=a["parent"],   # noqa: E731
                                          group=group, copies=a["copies"], ws=workspace(0))
    for page, group in ((BIG, 4), (16, BIG), (16, -1), (0, 4), (16, -2 ** 32 + 4)):
        with pytest.raises(sv.SVError):
            fork(page, group)
    wide = Strided(0, (12, 9), INT, (BIG + 9, 1))
    refused("sv_kv_fork", table=wide)
    refused("sv_kv_compact", table=wide)
    refused("sv_kv_compact", kept=Strided(0, (12, 6), INT, (BIG + 9, 1)))
    refused("sv_kv_copy", copies=On(0, (BIG, 3), INT))
    for shape in ((BIG, 16, 2, 64), (50, BIG, 2, 64), (50, 16, BIG, 64), (50, 16, 2, BIG)):
        refused("sv_kv_compact", pages=On(0, shape, torch.float16))
        refused("sv_kv_copy", layers=On(0, (5, *shape), torch.float16))
    refused("sv_kv_copy", layers=On(0, (BIG, 50, 16, 2, 64), torch.float16))
    assert made == []
    fork(16, 4)
    assert len(made) == 1
