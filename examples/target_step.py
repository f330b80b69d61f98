"""Speculative decoding of a one-layer toy target, every step on the device.

A step of a batch, as a serving loop runs it (with one layer instead of many):

  confidences -> sv.plan_budget           windows of the batch, packed by qo_indptr
  tokens      -> sv.kv_append             rotate queries and keys, append keys and values to the paged cache
              -> sv.paged_attention       every window over its request's cache
  logits      -> sv.verify_ragged         accept drafts, emit a token
  kv_len     += accepted drafts + 1       what was rejected is written over by the next window

Weights are random, so the text means nothing; the drafter guesses the target's next tokens with a chance it states as
its confidence.  Run: python examples/target_step.py [--requests 64] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_verification_rows_gb300 import sv  # noqa: E402


class Target:
    """Embedding, one attention layer over a paged cache, and the head."""

    def __init__(self, requests, max_len, K=7, vocab=4096, hq=16, hkv=4, d=64, page=16, interleaved=False, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        dt = torch.bfloat16

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[0] ** -0.5).to(dt)

        self.n, self.K, self.vocab, self.hq, self.hkv, self.d, self.page = requests, K, vocab, hq, hkv, d, page
        self.interleaved, self.device, self.width = interleaved, device, hq * d
        self.embed = torch.randn((vocab, self.width), generator=g, device=device).to(dt)
        self.w_qkv, self.w_out = weight(self.width, (hq + 2 * hkv) * d), weight(self.width, self.width)
        self.head = weight(self.width, vocab) * 8
        self.freq, self.mscale = sv.rotary_frequencies(d, scaling="yarn", factor=4.0, original_len=1024, device=device)
        per = -(-max_len // page)
        pages = torch.randperm(requests * per, generator=g, device=device).to(torch.int32)
        self.table = pages.view(requests, per).contiguous()
        self.k_pages = torch.zeros((requests * per, page, hkv, d), dtype=dt, device=device)
        self.v_pages = torch.zeros_like(self.k_pages)
        self.kv_len = torch.zeros(requests, dtype=torch.int32, device=device)      # committed tokens
        self.ws = sv.Workspace(device)

    def forward(self, tokens, qo_indptr, kv_len, max_window):
        """Logits [len(tokens), vocab] of packed windows that end at kv_len; rows past qo_indptr[-1] are padding."""
        x = self.embed[tokens.long()]
        qkv = (x @ self.w_qkv).view(-1, self.hq + 2 * self.hkv, self.d)
        q, k, v = qkv.split([self.hq, self.hkv, self.hkv], dim=1)                  # views of one projection
        q = sv.kv_append(k, v, self.k_pages, self.v_pages, self.table, qo_indptr, kv_len, self.freq, self.interleaved,
                         self.mscale, q=q)
        a = sv.paged_attention(q, self.k_pages, self.v_pages, self.table, qo_indptr, kv_len, max_window, lse=False,
                               ws=self.ws).out
        x = x + (a.reshape(-1, self.width) @ self.w_out)
        return x @ self.head

    def step(self, anchor, drafts, conf, budget, bucket, temperature, top_k, top_p, seed):
        """One verify step: (VerifyOut, verify_lens, qo_indptr, tokens, logits).  anchor [n]: the last emitted token,
        not yet in the cache; drafts [n, K]; conf [n, K]."""
        verify_lens, qo, _, _ = sv.plan_budget(conf, budget, bucket, ws=self.ws)
        block = torch.cat([anchor[:, None], drafts], dim=1)                        # [n, K + 1]
        row = torch.arange(bucket, dtype=torch.int32, device=self.device)
        r = (torch.searchsorted(qo, row, right=True) - 1).clamp(max=self.n - 1)
        at = (row - qo[r]).clamp(0, self.K)
        tokens = block[r, at.long()]                                               # padding rows repeat some token
        kv_len = self.kv_len + verify_lens + 1
        logits = self.forward(tokens, qo, kv_len, self.K + 1)
        out = sv.verify_ragged(logits, None, qo, verify_lens, drafts, temperature, top_k, top_p, seed=seed, ws=self.ws)
        self.kv_len += out.num_emitted                                             # accepted drafts and their anchor
        return out, verify_lens, qo, tokens, logits


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    n, K = a.requests, 7
    sv.load(build_if_missing=True)
    target = Target(n, max_len=(K + 1) * a.steps + 8, K=K)
    g = torch.Generator(device="cuda").manual_seed(1)
    budget = bucket = n * 5
    anchor = torch.randint(0, target.vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    greedy = torch.zeros(n, device="cuda")
    emitted = torch.zeros((), dtype=torch.int64, device="cuda")
    submitted = torch.zeros((), dtype=torch.int64, device="cuda")
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for s in range(a.steps):
        if s == 2:
            start.record()
        conf = 0.9 ** torch.arange(1, K + 1, device="cuda") * torch.rand((n, 1), generator=g, device="cuda").sqrt()
        drafts = torch.randint(0, target.vocab, (n, K), generator=g, device="cuda", dtype=torch.int32)
        out, lens, _, _, _ = target.step(anchor, drafts, conf.contiguous(), budget, bucket, greedy, None, None, s)
        anchor = out.out_tokens.gather(1, out.accept_len.long()[:, None]).squeeze(1)
        emitted += out.num_emitted.sum()
        submitted += (lens + 1).sum()
    stop.record()
    torch.cuda.synchronize()
    ms = start.elapsed_time(stop) / max(a.steps - 2, 1)
    print(f"{n} requests, {a.steps} steps: {int(emitted)} tokens emitted of {int(submitted)} verified, {ms:.3f} ms a step")


if __name__ == "__main__":
    main()
