"""The example's decoding loop: rotation, append, attention and verification together, against the same layer recomputed
from the tokens alone, with dense attention in fp32."""
import math
import os
import subprocess
import sys

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


def dense_logits(t, tokens):
    """The layer's logits at every position of one request's tokens, nothing cached."""
    x = t.embed[tokens.long()]
    qkv = (x @ t.w_qkv).view(-1, t.hq + 2 * t.hkv, t.d)
    q, k, v = qkv.split([t.hq, t.hkv, t.hkv], dim=1)
    p = torch.arange(len(tokens), device=x.device)
    turn = p.double()[:, None] * t.freq.double().sum(1)
    c, s = ((f(2 * math.pi * turn) * t.mscale)[:, None].float() for f in (torch.cos, torch.sin))

    def rotate(z):
        a, b = z.float().chunk(2, dim=-1)
        return torch.cat([a * c - b * s, b * c + a * s], dim=-1).to(torch.bfloat16).float()

    q, k, v = rotate(q), rotate(k).repeat_interleave(t.hq // t.hkv, 1), v.float().repeat_interleave(t.hq // t.hkv, 1)
    w = torch.einsum("qhd,khd->hqk", q, k) * t.d ** -0.5
    w = w.masked_fill(p[None, :] > p[:, None], -math.inf).softmax(-1)
    a = torch.einsum("hqk,khd->qhd", w, v).to(torch.bfloat16)
    return (x + a.reshape(-1, t.width) @ t.w_out) @ t.head


@pytest.mark.parametrize("d", [64, 128])
def test_a_decoding_loop_stays_on_the_dense_layers_logits(d):
    from target_step import Target
    n, K, steps = 6, 5, 9
    t = Target(n, max_len=80, K=K, vocab=512, hq=8, hkv=2, d=d)
    g = torch.Generator(device="cuda").manual_seed(3)
    anchor = torch.randint(0, 512, (n,), generator=g, device="cuda", dtype=torch.int32)
    text = [[int(x)] for x in anchor]
    greedy = torch.zeros(n, device="cuda")
    accepted = 0
    for s in range(steps):
        conf = torch.rand((n, K), generator=g, device="cuda")
        drafts = torch.randint(0, 512, (n, K), generator=g, device="cuda", dtype=torch.int32)
        if s:                                   # the drafter knows the first tokens of every other request's next window
            for r in range(0, n, 2):
                for j in range(2):
                    ids = torch.tensor(text[r] + drafts[r, :j].tolist(), device="cuda")
                    drafts[r, j] = dense_logits(t, ids)[-1].argmax()
        before = t.kv_len.tolist()
        out, lens, qo, tokens, logits = t.step(anchor, drafts, conf, n * 4, n * 4, greedy, None, None, s)
        for r in range(n):
            assert before[r] == len(text[r]) - 1                   # everything but the anchor is in the cache
            lo, hi = int(qo[r]), int(qo[r + 1])
            ids = torch.tensor(text[r][:-1] + tokens[lo:hi].tolist(), device="cuda")
            want = dense_logits(t, ids)[-(hi - lo):].float()
            # attention and the residual are rounded to bf16 at the same places on both sides; what differs are sums in
            # other orders: a few roundings of 2^-9 through a head of weights of size 8 / sqrt(width)
            assert (logits[lo:hi].float() - want).abs().max() <= 0.03 * want.abs().max()
            a = int(out.accept_len[r])
            assert out.out_tokens[r, :a].tolist() == drafts[r, :a].tolist()
            assert int(out.out_tokens[r, a]) == int(logits[lo + a].float().argmax())
            text[r] += out.out_tokens[r, :a + 1].tolist()
            accepted += a
        anchor = out.out_tokens.gather(1, out.accept_len.long()[:, None]).squeeze(1)
        assert t.kv_len.tolist() == [len(x) - 1 for x in text]
    assert accepted > steps                                         # drafts were accepted, and their slots kept


def test_the_step_is_captured_in_a_graph():
    from target_step import Target
    n, K = 4, 3
    t = Target(n, max_len=64, K=K, vocab=256, hq=4, hkv=2, d=64)
    g = torch.Generator(device="cuda").manual_seed(5)
    anchor = torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.int32)
    drafts = torch.randint(0, 256, (n, K), generator=g, device="cuda", dtype=torch.int32)
    conf, greedy = torch.rand((n, K), generator=g, device="cuda"), torch.zeros(n, device="cuda")
    step = lambda: t.step(anchor, drafts, conf, 12, 12, greedy, None, None, 0)   # noqa: E731
    step()
    t.kv_len.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    t.kv_len.zero_()
    graph.replay()
    torch.cuda.synchronize()
    tokens, logits = out[0].out_tokens.clone(), out[4].clone()
    t.kv_len.zero_()
    want = step()
    assert torch.equal(tokens, want[0].out_tokens) and torch.equal(logits, want[4])


def test_the_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "target_step.py"), "--requests", "8", "--steps", "6"],
                       capture_output=True, text=True, timeout=200)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "tokens emitted" in r.stdout
