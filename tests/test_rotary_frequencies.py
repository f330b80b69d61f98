"""The frequency tables of the rotation, and what the attention calls refuse on the host (no GPU)."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    sv_build.build()
    return sv.load()


def radians(freq):
    return freq.double().sum(1) * 2 * math.pi


@pytest.mark.parametrize("rot", [2, 10, 64, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_plain_frequencies_are_powers_of_the_base(rot, base):
    freq, mscale = sv.rotary_frequencies(rot, base, device="cpu")
    assert freq.shape == (rot // 2, 2) and freq.dtype == torch.float32 and mscale == 1.0
    for m, f in enumerate(radians(freq).tolist()):
        assert f == pytest.approx(base ** (-2 * m / rot), rel=2.0 ** -45)   # high + low carries 48 bits


def test_linear_and_ntk_scaling():
    plain = radians(sv.rotary_frequencies(64, device="cpu")[0])
    assert torch.allclose(radians(sv.rotary_frequencies(64, scaling="linear", factor=4.0, device="cpu")[0]), plain / 4,
                          rtol=1e-12, atol=0)
    ntk = radians(sv.rotary_frequencies(64, scaling="ntk", factor=4.0, device="cpu")[0])
    assert float(ntk[0]) == pytest.approx(1.0, rel=1e-13)
    assert float(ntk[-1]) == pytest.approx(float(plain[-1]) / 4, rel=1e-12)   # base' makes the slowest pair 4x slower


def test_yarn_keeps_fast_pairs_divides_slow_ones_and_scales():
    plain = radians(sv.rotary_frequencies(128, device="cpu")[0])
    freq, mscale = sv.rotary_frequencies(128, scaling="yarn", factor=8.0, original_len=4096, device="cpu")
    ratio = radians(freq) / plain
    # correction dimension of b turns: 128 ln(4096 / (2 pi b)) / (2 ln 10000)
    low = math.floor(128 * math.log(4096 / (2 * math.pi * 32)) / (2 * math.log(10000)))
    high = math.ceil(128 * math.log(4096 / (2 * math.pi)) / (2 * math.log(10000)))
    for m in range(64):
        ramp = min(max((m - low) / (high - low), 0), 1)
        assert float(ratio[m]) == pytest.approx(1 - ramp + ramp / 8, rel=1e-12), m
    assert mscale == pytest.approx(0.1 * math.log(8) + 1)


def test_bands_keep_short_wavelengths_and_divide_long_ones():
    plain = radians(sv.rotary_frequencies(128, 500000.0, device="cpu")[0])
    freq, mscale = sv.rotary_frequencies(128, 500000.0, scaling="bands", factor=8.0, original_len=8192, device="cpu")
    assert mscale == 1.0
    for f, p in zip(radians(freq).tolist(), plain.tolist()):
        wave = 2 * math.pi / p
        if wave < 8192 / 4:
            want = p
        elif wave > 8192:
            want = p / 8
        else:
            s = (8192 / wave - 1) / 3
            want = (1 - s) * p / 8 + s * p
        assert f == pytest.approx(want, rel=1e-12)


def test_frequency_refusals():
    for kw in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=8, factor=0.0), dict(rot_dim=8, base=1.0),
               dict(rot_dim=8, scaling="yarn", factor=2.0), dict(rot_dim=8, scaling="other")):
        with pytest.raises(sv.SVError):
            sv.rotary_frequencies(device="cpu", **kw)


def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "sv.h"\n'
                   "int main(void) {\n"
                   '  printf("%zu %zu\\n", sizeof(sv_heads_t), offsetof(sv_heads_t, heads));\n'
                   '  printf("%zu %zu %zu\\n", sizeof(sv_paged_kv_t), offsetof(sv_paged_kv_t, page_table),\n'
                   "         offsetof(sv_paged_kv_t, page_size));\n"
                   '  printf("%zu %zu\\n", sizeof(sv_rotary_t), offsetof(sv_rotary_t, mscale));\n'
                   '  printf("%d %d %d %d\\n", (int)SV_ROTARY_INTERLEAVED, (int)SV_ROTARY_INVERSE, (int)SV_ATTN_FULL,\n'
                   "         (int)SV_DTYPE_F16);\n"
                   "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [[int(x) for x in line.split()] for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                                     check=True).stdout.strip().split("\n")]
    assert got[0] == [ctypes.sizeof(sv.Heads), sv.Heads.heads.offset]
    assert got[1] == [ctypes.sizeof(sv.PagedKV), sv.PagedKV.page_table.offset, sv.PagedKV.page_size.offset]
    assert got[2] == [ctypes.sizeof(sv.RotaryArgs), sv.RotaryArgs.mscale.offset]
    assert got[3] == [sv.ROTARY_INTERLEAVED, sv.ROTARY_INVERSE, sv.ATTN_FULL, sv.DTYPE_F16]


FAKE = 0x1000   # never dereferenced: the checks fail first


def heads(n, data=FAKE):
    return sv.Heads(data, 1024, 128, n)


def cache(n=2, page_size=16, max_pages=4, ld=4, data=FAKE, v_heads=None, n_pages=8):
    return sv.PagedKV(heads(n, data), heads(n if v_heads is None else v_heads, data), 4096, 4096, FAKE, ld, max_pages,
                      n_pages, page_size)


def rope(rot=64, freq=FAKE, flags=0):
    return sv.RotaryArgs(freq, rot, flags, 1.0)


def test_rotary_argument_errors(lib):
    def call(x=heads(4), y=heads(4, 0x2000), dt=0, tokens=3, d=128, pos=FAKE, r=rope()):
        return lib.sv_rotary(x, y, dt, tokens, d, pos, r, None)
    assert call(x=heads(4, None)) == sv.SV_ERR_INVALID_ARG
    assert call(y=heads(4, None)) == sv.SV_ERR_INVALID_ARG
    assert call(pos=None) == sv.SV_ERR_INVALID_ARG
    assert call(tokens=-1) == sv.SV_ERR_INVALID_ARG
    assert call(dt=3) == sv.SV_ERR_INVALID_ARG
    assert call(y=heads(5, 0x2000)) == sv.SV_ERR_INVALID_ARG
    assert call(r=rope(rot=63)) == sv.SV_ERR_INVALID_ARG
    assert call(r=rope(rot=130)) == sv.SV_ERR_INVALID_ARG
    assert call(r=rope(freq=None)) == sv.SV_ERR_INVALID_ARG
    assert call(d=257) == sv.SV_ERR_UNSUPPORTED
    assert call(y=sv.Heads(FAKE, 2048, 128, 4)) == sv.SV_ERR_INVALID_ARG     # in place with other strides
    assert call(tokens=0, x=heads(4, None)) == sv.SV_OK                      # nothing to do


def test_append_argument_errors(lib):
    none = heads(0, None)

    def call(k=heads(2), v=heads(2), c=cache(), dt=0, tokens=3, d=128, n=2, qo=FAKE, kv=FAKE, r=rope(), q=none, o=none):
        return lib.sv_kv_append(k, v, c, dt, tokens, d, n, qo, kv, r, q, o, None, None)
    assert call(k=heads(2, None)) == sv.SV_ERR_INVALID_ARG
    assert call(v=heads(3)) == sv.SV_ERR_INVALID_ARG
    assert call(c=cache(n=3)) == sv.SV_ERR_INVALID_ARG
    assert call(c=cache(page_size=0)) == sv.SV_ERR_INVALID_ARG
    assert call(c=cache(ld=3)) == sv.SV_ERR_INVALID_ARG
    assert call(c=cache(data=None)) == sv.SV_ERR_INVALID_ARG
    assert call(n=0) == sv.SV_ERR_INVALID_ARG
    assert call(qo=None) == sv.SV_ERR_INVALID_ARG
    assert call(r=rope(flags=sv.ROTARY_INVERSE)) == sv.SV_ERR_INVALID_ARG
    assert call(q=heads(4)) == sv.SV_ERR_INVALID_ARG                          # q without q_out
    assert call(d=512, r=rope()) == sv.SV_ERR_UNSUPPORTED
    assert call(tokens=0) == sv.SV_OK


def test_attention_argument_errors(lib):
    def call(q=heads(8), c=cache(), dt=0, tokens=3, d=128, n=2, qo=FAKE, kv=FAKE, mw=2, scale=0.1, win=0, flags=0,
             o=heads(8, 0x8000), ws=0x100000, ws_bytes=1 << 40):
        return lib.sv_paged_attention(q, c, dt, tokens, d, n, qo, kv, mw, scale, win, flags, o, None, None, ws, ws_bytes,
                                      None)
    assert call(q=heads(8, None)) == sv.SV_ERR_INVALID_ARG
    assert call(o=heads(8, None)) == sv.SV_ERR_INVALID_ARG
    assert call(o=heads(6, 0x8000)) == sv.SV_ERR_INVALID_ARG
    assert call(q=heads(7), o=heads(7, 0x8000)) == sv.SV_ERR_INVALID_ARG     # 7 heads over 2 key heads
    assert call(c=cache(v_heads=3)) == sv.SV_ERR_INVALID_ARG
    assert call(c=cache(max_pages=-1)) == sv.SV_ERR_INVALID_ARG
    assert call(dt=5) == sv.SV_ERR_INVALID_ARG
    assert call(win=-1) == sv.SV_ERR_INVALID_ARG
    assert call(mw=-1) == sv.SV_ERR_INVALID_ARG
    assert call(scale=math.inf) == sv.SV_ERR_INVALID_ARG
    assert call(scale=math.nan) == sv.SV_ERR_INVALID_ARG
    assert call(kv=None) == sv.SV_ERR_INVALID_ARG
    assert call(d=257) == sv.SV_ERR_UNSUPPORTED
    assert call(ws=None) == sv.SV_ERR_WORKSPACE
    assert call(ws=0x100001) == sv.SV_ERR_WORKSPACE
    assert call(ws_bytes=16) == sv.SV_ERR_WORKSPACE
    assert call(tokens=0, ws=None) == sv.SV_OK
    assert lib.sv_attention_workspace_size(4, 8, 3, 128) == 0
    assert lib.sv_attention_workspace_size(4, 8, 2, 512) == 0
    assert lib.sv_attention_workspace_size(4, 8, 2, 128) > 0


def test_the_calls_refuse_host_tensors():
    x, i = torch.zeros((2, 4, 8)), torch.zeros(2, dtype=torch.int32)
    pages, table = torch.zeros((2, 4, 4, 8)), torch.zeros((2, 1), dtype=torch.int32)
    with pytest.raises(sv.SVError):
        sv.rotary(x, i, torch.zeros((4, 2)))
    with pytest.raises(sv.SVError):
        sv.kv_append(x, x, pages, pages, table, torch.zeros(3, dtype=torch.int32), i)
    with pytest.raises(sv.SVError):
        sv.paged_attention(x, pages, pages, table, torch.zeros(3, dtype=torch.int32), i, 1)
