"""Which kernel each size of kernel_cases.py gets, asked of the library on the
CPU: a change of the rules may not leave a kernel without a test."""
import os
import re
import shutil
import subprocess

import pytest

from kernel_cases import CASES
from mixed_precision_weight_page_amd import pagedweight as pwb

HERE = os.path.dirname(os.path.abspath(__file__))
TYPES = {"DF16b": "bf16", "DF16_": "f16", "4E4M3": "e4m3", "8E4M3Full": "e4m3 full"}
DT = {"f32": 0, "f16": 1, "bf16": 2, "e4m3": 3}


def read(name):
    """(kernel, operands, SwiGLU, grouped) of a mangled name, None for other kernels."""
    m = re.search(r"\d\d?(product_\w+?|fp8_skinny)_kernelI(?:NS\d?_)?(DF16b|DF16_|4E4M3|8E4M3Full)E?((?:Li\d+E)*)((?:Lb\dE)+)E", name)
    if not m:
        return None
    n, b = [int(v) for v in re.findall(r"Li(\d+)", m.group(3))], [v == "1" for v in re.findall(r"Lb(\d)", m.group(4))]
    kind = m.group(1).replace("product_", "")
    kernel = {"phased": lambda: "phased", "ring": lambda: f"ring {n[0]}x{n[1]}/{n[4]}", "any": lambda: f"any {n[0]}",
              "stream": lambda: f"stream {n[0]}x{n[1]}", "fp8_skinny": lambda: "skinny"}[kind]()
    return kernel, TYPES[m.group(2)], b[0], len(b) > 1 and b[1]


def line(c):
    size, cols = {"e4m3": 1}.get(c.dtype, 2), c.K
    full = (c.M, c.N, c.K, 6 if c.glu else 0, DT[c.out], cols + c.pads[0], cols + c.pads[1])
    assert size == 1 or c.dtype in ("bf16", "f16")
    return " ".join(map(str, full + ((len(c.counts), DT[c.dtype], 1 if c.tokens else 0) if c.counts else ())))


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    if not shutil.which("gcc") or not os.path.exists(pwb.library_path()):
        pytest.skip("no gcc or no library")
    probe = str(tmp_path_factory.mktemp("probe") / "launch_probe")
    subprocess.run(["gcc", "-O1", "-rdynamic", "-I", os.path.join(HERE, "..", "include"), os.path.join(HERE, "launch_probe.c"),
                    "-o", probe, "-ldl"], check=True)
    r = subprocess.run([probe, pwb.library_path()], input="\n".join(map(line, CASES)) + "\n", capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr
    out = r.stdout.splitlines()
    return [v[4:] for v in out if v.startswith("has ")], [v for v in out if not v.startswith("has ")]


def test_every_size_gets_its_kernel(answers):
    got = answers[1]
    assert len(got) == len(CASES)
    wrong = []
    for c, g in zip(CASES, got):
        full = c.dtype == "e4m3" and c.out == "f32"
        want = (c.kernel, c.dtype + (" full" if full else ""), c.glu, c.counts is not None)
        if read(g.split()[0]) != want:
            wrong.append((c.name, read(g.split()[0]) or g))
    assert not wrong


def test_every_kernel_has_a_size(answers):
    there = {read(n) for n in answers[0]} - {None}
    assert len(there) == 118
    assert there == {read(g.split()[0]) for g in answers[1]}
