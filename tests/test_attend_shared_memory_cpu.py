"""The few-rows attention counts on two CTAs an SM: what nvcc reports of each variant's shared memory has to leave room."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SM, EACH = 228 * 1024, 1024        # bytes of an SM, and what the system takes for each CTA


def test_two_ctas_fit_an_sm(tmp_path):
    from speculative_decoding_verify_07_gb300 import build
    source = open(os.path.join(build.CSRC, "spec_attend_rows.cu")).read()
    probe = tmp_path / "shapes.cu"
    shapes = [(d, e, m) for d in (64, 128) for e in (0, 1) for m in (1, 2)]
    probe.write_text(source + "\n#include <cstdio>\nint main() {\n" + "\n".join(
        f'  printf("%d\\n", (int)specv::RowsShape<{d}, {"true" if e else "false"}, {m}>::smem);' for d, e, m in shapes) + "\n}\n")
    run = subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-Xptxas", "-v", "-I", build.CSRC, "-o", str(tmp_path / "shapes"),
                          str(probe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    fixed = {}
    for kernel, used in re.findall(r"Compiling entry function '([^']+)'.*?\n.*?Used ([^\n]+)", run.stderr, re.S):
        d, e, m = re.search(r"attend_rows_kernelILi(\d+)ELb(\d)ELi(\d)E", kernel).groups()
        fixed[int(d), int(e), int(m)] = int(re.search(r"(\d+) bytes smem", used)[1])
    dynamic = subprocess.run([str(tmp_path / "shapes")], capture_output=True, text=True).stdout.split()
    assert sorted(fixed) == shapes and len(dynamic) == len(shapes)
    over = {s: fixed[s] + int(n) for s, n in zip(shapes, dynamic) if 2 * (fixed[s] + int(n) + EACH) > SM}
    assert not over, over
