"""The block norm replaces v / scale by a reciprocal and one correction step
for its fp32 values.  tests/quantize_fp32_division_check.c compares the codes
next to every boundary between two of them, for random row maxima."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_values_next_to_a_boundary_get_the_code_of_the_division(tmp_path):
    exe = str(tmp_path / "check")
    subprocess.run(["gcc", "-O2", "-mfma", "-ffp-contract=off", "-std=c11",
                    os.path.join(ROOT, "tests", "quantize_fp32_division_check.c"), "-o", exe, "-lm"], check=True)
    parts = [subprocess.Popen([exe, "100000", str(i)], stdout=subprocess.PIPE, text=True) for i in range(4)]
    outs = [p.communicate(timeout=600)[0] for p in parts]
    assert all(p.returncode == 0 for p in parts), outs
    assert sum(int(o) for o in outs) > 500_000_000     # of 7.1e8, less what lies past the maximum
