"""The large tiles of the dense product wait for copies by their number
(s_waitcnt vmcnt), so the emitted code has to issue them in the order the
waits count on: a stage's 16-byte copies to LDS first, the 4-byte load that
asks for a later stage last. Checked in the compiler's output for gfx950."""
import os
import re
import shutil
import subprocess

import pytest

from mixed_precision_weight_page_amd import build


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not shutil.which("hipcc"):
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("asm") / "linear.s"
    r = subprocess.run(["hipcc", *build.COMMON, "--cuda-device-only", "-S", os.path.join(build.CSRC, "kernels_linear.hip"),
                        "-o", str(out)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    found, name = {}, None
    for line in out.read_text().splitlines():
        label = re.match(r"(_Z\S+):", line)
        if label:
            name = label.group(1)
        wait = re.search(r"s_waitcnt.*vmcnt\((\d+)\)", line)
        what = ("copy" if re.search(r"buffer_load_dwordx4 .*\blds\b", line) else
                "touch" if re.search(r"buffer_load_dword .*\blds\b", line) else
                "load" if re.search(r"\b(global|buffer|flat|scratch)_(load|store)", line) else
                int(wait.group(1)) if wait else None)
        if name and what is not None:
            found.setdefault(name, []).append(what)
    return found


def test_stages_of_the_large_tiles_are_issued_in_order(kernels):
    phased = {n: seq for n, seq in kernels.items() if "linear_phased_kernel" in n}
    assert len(phased) == 8   # two tiles, SwiGLU or not, bf16 and fp16
    for name, seq in phased.items():
        copies = 8 if "Li8E" in name else 7   # 64-row parts of a stage: (256 or 192) + 256 rows
        # stage 0, three early loads, the wait that leaves those; then per
        # stage its copies, one early load, the waits that leave that one
        want = ["copy"] * copies + ["touch"] * 3 + [3] + ["copy"] * copies + ["touch"] + [1, 1, 0]
        assert seq[:len(want)] == want, (name, seq[:len(want) + 4])
        assert "touch" not in seq[len(want):] and "copy" not in seq[len(want):], name
