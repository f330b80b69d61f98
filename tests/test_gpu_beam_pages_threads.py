"""Beam and page calls of several threads at once, each with its own stream, workspace and tensors, from a process's first
call on."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import sv
from tests.beam_cases import Pool, select64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
THREADS, TURNS = 6, 20

pytestmark = pytest.mark.gpu


def work(seed, ready, failed):
    try:
        g = torch.Generator().manual_seed(seed)
        n, beams, vocab, n_out = (3, 4, 5001, 8) if seed % 2 else (60, 3, 3001, 6)
        logits = torch.randn((n, beams, vocab), generator=g) * 3
        scores = -torch.rand((n, beams), generator=g)
        tokens, parents, _ = select64(logits, scores, n_out)
        requests = 40 + seed if seed % 3 else 1040
        pool = Pool(requests, 8, 9 * requests, 16)
        stream, ws = torch.cuda.Stream(), sv.Workspace("cuda")
        with torch.cuda.stream(stream):
            x, c, on = logits.cuda(), scores.cuda(), pool.gpu()
            keep, room = (torch.full((requests,), v, dtype=torch.int32, device="cuda") for v in (0, 100))
            stream.synchronize()
            ready.wait(60)
            out = [sv.beam_select(x, c, n_out, ws=ws) for _ in range(TURNS)]
            for _ in range(TURNS):
                sv.kv_fork(*on, 16, keep, room, ws=ws)
            stream.synchronize()
            for o in out:
                assert torch.equal(o.tokens.cpu(), tokens) and torch.equal(o.parents.cpu(), parents)
            pool.fork([0] * requests, [100] * requests)
            for a, b in zip(on, (pool.table, pool.held, pool.ref)):
                assert torch.equal(a.cpu(), b)
    except BaseException as e:                      # a thread's failure is the process's
        failed.append(repr(e))
        raise


def main():
    ready, failed = threading.Barrier(THREADS), []
    threads = [threading.Thread(target=work, args=(s, ready, failed), daemon=True) for s in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(100)
    assert not failed and not any(t.is_alive() for t in threads), failed
    print("threads: ok")


def test_threads_call_at_once():
    r = subprocess.run([sys.executable, "-c", "from tests.test_gpu_beam_pages_threads import main; main()"], cwd=ROOT,
                       capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "threads: ok" in r.stdout, r.stderr[-2000:]
