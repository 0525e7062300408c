"""As test_product_order.py, for the kernels of e4m3 products with an fp32 y:
the emitted code issues a step's copies together and in the order of the
steps, and keeps nothing in scratch memory."""
import os
import re
import shutil
import subprocess

import pytest

from mixed_precision_weight_page_amd import build

SOURCES = ("kernels_fp8_full.hip", "kernels_grouped8_full.hip")
WHAT = (("copy", r"buffer_load_dwordx4 .*\blds\b"), ("scale", r"buffer_load_dword .*\blds\b"), ("scratch", r"\bscratch_(load|store)"),
        ("load", r"\b(global|buffer|flat)_(load|store)"), ("mfma8", r"v_mfma_\S*f8f6f4"), ("mfma", r"v_mfma"))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """name -> its copies, other memory and matrix instructions, and waits, in order."""
    if not shutil.which("hipcc"):
        pytest.skip("no hipcc")
    found, folder = {}, tmp_path_factory.mktemp("asm")
    runs = [subprocess.Popen(["hipcc", *build.COMMON, "--cuda-device-only", "-S", os.path.join(build.CSRC, s), "-o", str(folder / s)],
                             stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True) for s in SOURCES]
    for s, r in zip(SOURCES, runs):
        err = r.communicate(timeout=600)[1]
        assert r.returncode == 0, err[-2000:]
        name = None
        for line in (folder / s).read_text().splitlines():
            label = re.match(r"(_Z\S+):", line)
            name = label.group(1) if label else name
            wait = re.search(r"s_waitcnt.*vmcnt\((\d+)\)", line)
            what = int(wait.group(1)) if wait else next((w for w, p in WHAT if re.search(p, line)), None)
            if name and what is not None:
                found.setdefault(name, []).append(what)
    return found


def test_nothing_is_cut_off_or_kept_in_scratch(kernels):
    products = {n: seq for n, seq in kernels.items() if "mfma" in seq or "mfma8" in seq}
    assert len(products) == 2 * (4 + 2 + 4 + 1) + 2 * (4 + 2 + 2) - 1   # with SwiGLU no block of 16 weight rows alone
    for name, seq in products.items():
        assert "mfma8" not in seq and "scratch" not in seq, name


def test_ring_steps_are_issued_in_order(kernels):
    seen = 0
    for name, seq in kernels.items():
        m = re.search(r"product_ring_kernelI\S*?Li(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb", name)
        if not m:
            continue
        bm, bn, wm, wn, d = map(int, m.groups())
        step = sorted(["copy"] * ((bm + bn) // 8 // (wm * wn)) + ["scale"])
        n = len(step)
        body = seq[seq.index("copy"):]
        for j in range(d - 1):
            assert sorted(map(str, body[j * n:(j + 1) * n])) == step, (name, j, body[:60])
        rest = [w for w in body[(d - 1) * n:] if w != 0]
        assert rest[0] == (d - 2) * n or (d == 2 and rest[0] != 0), (name, rest[:20])
        rest = rest[1:] if d > 2 else rest
        assert sorted(map(str, rest[:n])) == step, (name, rest[:20])
        assert "mfma" in rest[n:n + 2] and not {"copy", "scale"} & set(rest[n:]), name
        seen += 1
    assert seen == 4 * 2 * 2   # tiles; SwiGLU or not; dense and grouped


def test_stream_pieces_are_issued_in_order(kernels):
    seen = 0
    for name, seq in kernels.items():
        m = re.search(r"product_stream_kernelI\S*?Li(\d+)ELi(\d+)ELi(\d+)ELb", name)
        if not m:
            continue
        rb, mb, d = map(int, m.groups())
        step = sorted(["copy"] * (2 * (rb + mb)) + ["scale"] * 2)
        n = len(step)
        body = seq[seq.index("copy"):]
        for j in range(d):
            assert sorted(map(str, body[j * n:(j + 1) * n])) == step, (name, j, body[:60])
        rest = [w for w in body[d * n:] if w in ("copy", "scale", "load", 0, (d - 1) * n)]
        at = rest.index((d - 1) * n)
        after = rest[at + 1:]
        end = next(i for i, w in enumerate(after) if w not in ("copy", "scale"))
        assert sorted(map(str, rest[:at] + after[:end])) == step, (name, rest[:40])
        seen += 1
    assert seen
