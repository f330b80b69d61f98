"""The attention operators' binding runs the library on the device that the tensors live on, whichever is current.  On the
host: tensors and the library are stand-ins that record what is asked of them."""
import contextlib
import types

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import sv


class On:
    """As much of a contiguous GPU tensor as the binding looks at."""

    is_cuda = True

    def __init__(self, device, shape, dtype):
        self.n, self.shape, self.dtype, self.device = device, torch.Size(shape), dtype, torch.device("cuda", device)

    def get_device(self):
        return self.n

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


@pytest.fixture
def calls(monkeypatch):
    """(entry, device that was current) of every call of the library."""
    made, current = [], [0]

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(sv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(sv, "attention_workspace_size", lambda *sizes: 1024)
    entry = lambda name: lambda *a: made.append((name, current[0])) or 0   # noqa: E731
    names = ("sv_rotary", "sv_kv_append", "sv_paged_attention")
    monkeypatch.setattr(sv, "_lib", types.SimpleNamespace(**{x: entry(x) for x in names}))
    return made


def tensors(device):
    heads = lambda n: On(device, (4, n, 64), torch.bfloat16)               # noqa: E731
    ints = lambda *shape: On(device, shape, torch.int32)                   # noqa: E731
    pages = On(device, (6, 16, 2, 64), torch.bfloat16)
    return dict(q=heads(4), out=heads(4), k=heads(2), pages=pages, table=ints(2, 3), qo=ints(3), lens=ints(2), pos=ints(4),
                freq=On(device, (32, 2), torch.float32))


def workspace(device):
    ws = sv.Workspace("cuda")
    ws.buf = On(device, (4096,), torch.uint8)
    return ws


def run_all(t, ws):
    sv.rotary(t["q"], t["pos"], t["freq"], out=t["out"])
    sv.kv_append(t["k"], t["k"], t["pages"], t["pages"], t["table"], t["qo"], t["lens"], t["freq"], q=t["q"], q_out=t["out"])
    sv.paged_attention(t["q"], t["pages"], t["pages"], t["table"], t["qo"], t["lens"], 4, out=t["out"], lse=False, ws=ws)


@pytest.mark.parametrize("device", [0, 1, 3])
def test_the_library_runs_on_the_tensors_device(calls, device):
    run_all(tensors(device), workspace(device))
    assert calls == [("sv_rotary", device), ("sv_kv_append", device), ("sv_paged_attention", device)]
    assert torch.cuda.current_device() == 0


def test_a_workspace_on_another_device_is_refused(calls):
    with pytest.raises(sv.SVError, match="cuda:1"):
        run_all(tensors(1), workspace(0))
    assert [x for x, _ in calls] == ["sv_rotary", "sv_kv_append"]


def test_tensors_on_two_devices_are_refused(calls):
    t = tensors(1)
    for name in ("k", "pages", "table", "qo", "lens"):
        with pytest.raises(sv.SVError):
            u = dict(t, **{name: tensors(0)[name]})
            run_all(u, workspace(1))
    assert all(device == 1 for _, device in calls)
