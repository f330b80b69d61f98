"""The status bits of sv.h and of the binding are the same, and every refusal is among the errors."""
import os
import re
import subprocess

from speculative_decoding_verification_rows_gb300 import sv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INFORMATIONAL = {"Q_ZERO", "RESID_ZERO"}


def test_the_bits_and_the_mask_of_errors(tmp_path):
    with open(os.path.join(ROOT, "include", "sv.h")) as f:
        names = re.findall(r"^    SV_ROW_(\w+) = \d+", f.read(), re.M)
    assert len(names) == 10 and INFORMATIONAL < set(names)
    src = tmp_path / "bits.c"
    prints = "".join(f'  printf("%d\\n", (int)SV_ROW_{x});\n' for x in names + ["ERROR_MASK"])
    src.write_text(f'#include <stdio.h>\n#include "sv.h"\nint main(void) {{\n{prints}  return 0;\n}}\n')
    exe = tmp_path / "bits"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    *bits, mask = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert bits == [getattr(sv, f"SV_ROW_{x}") for x in names] == [getattr(sv, f"ROW_{x}") for x in names]
    # a caller that looks at the mask alone must not take a refused request for one that was served
    assert mask == sv.ROW_ERROR_MASK == sum(b for x, b in zip(names, bits) if x not in INFORMATIONAL)
