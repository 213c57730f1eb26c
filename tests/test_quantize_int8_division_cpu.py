"""The int8 token quantiser replaces x / scale by a reciprocal and one
correction step for bf16 and fp16 rows.  tests/quantize_int8_division_check.c
compares the codes of both quotients for every pair of a magnitude and a row
maximum of either type (about 5e8 pairs each)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype,least", [("bf16", 530_000_000), ("fp16", 500_000_000)])
def test_every_pair_gets_the_code_of_the_division(tmp_path, dtype, least):
    exe = str(tmp_path / "check")
    subprocess.run(["gcc", "-O2", "-mfma", "-ffp-contract=off", "-std=c11",
                    os.path.join(ROOT, "tests", "quantize_int8_division_check.c"), "-o", exe, "-lm"], check=True)
    parts = [subprocess.Popen([exe, dtype, str(i), "4"], stdout=subprocess.PIPE, text=True) for i in range(4)]
    outs = [p.communicate(timeout=600)[0] for p in parts]
    assert all(p.returncode == 0 for p in parts), outs
    assert sum(int(o) for o in outs) > least
