"""Sizes for each kernel of the e4m3 and grouped products, and the kernel that
the rules give each of them: test_kernel_choice.py asks the library (on the
CPU) whether they still do, test_gpu_kernels.py computes them.

Kernels: "phased"; "ring R x C / D" (rows of x, weight rows, slots); "any R"
(rows of any alignment); "stream R x C" (blocks of 16 weight rows, of rows of x);
"skinny". A case's kernel stands with the type of its operands, whether it is
SwiGLU and whether it is grouped."""
from typing import NamedTuple, Optional, Tuple


class Case(NamedTuple):
    kernel: str
    M: int                       # rows (grouped: in all)
    N: int
    K: int
    out: str = "bf16"            # of e4m3 operands: "f32" is another kernel's
    glu: bool = False
    dtype: str = "e4m3"
    counts: Optional[Tuple[int, ...]] = None   # of each expert: grouped
    tokens: int = 0              # rows of x are gathered from so many
    pads: Tuple[int, int] = (0, 0)             # elements between rows of x, of w

    @property
    def name(self):
        c = self
        return (f"{c.kernel.replace(' ', '')}-{'grouped-' if c.counts else ''}{c.dtype}-{c.out}-{'swiglu-' if c.glu else ''}"
                f"{c.M}x{c.N}x{c.K}" + (f"-pads{c.pads[0]}_{c.pads[1]}" if any(c.pads) else "") + ("-rows" if c.tokens else ""))


def _dense():
    both = []
    # last tiles of 1 to 4 blocks of 64 rows; one step of K, two, three and more
    for M in (7200, 7239, 7300, 7400):
        both.append(("phased", M, 1800, 272, ("bf16",)))
    both += [("phased", 7239, 1803, 400, ("f16",)), ("phased", 12000, 3900, 128, ("f16",)), ("phased", 12000, 3900, 144, ("bf16",))]
    both += [("ring 128x128/2", 1290, 2980, 272, ("bf16",)), ("ring 128x128/4", 4500, 640, 272, ("f16",)),
             ("ring 128x256/3", 2048, 4096, 4096, ("bf16",)), ("ring 64x64/4", 40, 4900, 272, ("bf16",)),
             ("ring 128x128/2", 7030, 550, 272, ("f32",)), ("ring 128x128/4", 4540, 650, 272, ("f32",)),
             ("ring 128x256/3", 2580, 2940, 4096, ("f32",)), ("ring 64x64/4", 40, 4600, 272, ("f32",))]
    both += [("stream 2x1", 5, 9500, 528, ("bf16", "f32")), ("stream 2x2", 20, 5000, 272, ("f16", "f32")),
             ("stream 2x4", 110, 4090, 4096, ("bf16", "f32"))]
    for kernel, M, N, K, outs in both:
        for out in outs:
            yield Case(kernel, M, N, K, out)
            yield Case(kernel, M, N // 2, K, out, True)
    for out in ("bf16", "f32"):
        yield Case("stream 1x1", 3, 70, 4096, out)
        yield Case("stream 2x1", 3, 70, 4096, out, True)
        # row starts at all four residues of 4, K of whole steps and not
        for pads in ((0, 0), (1, 2), (2, 3), (3, 1)):
            for glu in (False, True):
                yield Case("skinny", 20, 310, 1167, out, glu, pads=pads)
                yield Case("any 64", 90, 2200, 165, out, glu, pads=pads)
                yield Case("any 128", 1700, 950 if glu else 1900, 261, out, glu, pads=pads)
        yield Case("any 128", 1700, 1900, 256, out, pads=(4, 4))   # rows at words, not at 16 bytes
        yield Case("skinny", 1, 40, 5, out)


def _grouped():
    spread = lambda M, E: tuple(M // E + (1 if e < M % E else 0) for e in range(E))  # noqa: E731
    for dtype in ("e4m3", "bf16", "f16"):
        for glu in (False, True):
            half = 2 if glu else 1
            put = lambda kernel, counts, N, K, out="bf16", **kw: Case(  # noqa: E731
                kernel, sum(counts), N // half, K, out, glu, dtype, tuple(counts), **kw)
            # last tiles of 1 to 4 blocks of 64 rows
            yield put("phased", (3100, 2160, 1330, 650), 6000, 400, tokens=900)
            yield put("phased", (3904, 0, 3335), 4100, 528, "f16" if dtype != "bf16" else "f32")
            yield put("ring 64x64/4", (30, 0, 41, 1), 200, 400, tokens=33)
            for out in ("bf16", "f32") if dtype == "e4m3" else ("bf16",):
                yield put("stream 2x1", (1, 0, 9, 3), 300, 272, out)
                yield put("stream 2x2", (30, 2, 0, 5), 300, 528, out, tokens=20)
                for pads in ((0, 0), (1, 2), (2, 3), (3, 1)):
                    yield put("any 64", (40, 3, 0, 70), 300, 165, out, pads=pads)
                    yield put("any 128", (1100, 1300), 1300, 261, out, pads=pads, tokens=500 if pads[0] else 0)
            if dtype != "e4m3":
                yield put("stream 4x1", (1, 0, 9, 3), 300, 528)
                yield put("ring 128x128/2", spread(800, 32), 2300 if not glu else 3200, 272)
                yield put("ring 128x128/4", (391, 700, 900, 500), 1100, 272)
                yield put("ring 128x256/3", (900, 20, 0, 800, 900), 2400, 528, tokens=300)
            else:
                yield put("ring 128x128/2", spread(800, 20), 2500, 272)
                yield put("ring 128x128/4", (5000, 2300), 350, 272)
                yield put("ring 128x256/3", (300, 300, 207), 8100, 4096)
                yield put("ring 64x64/4", (30, 0, 41, 1), 200, 400, "f32", tokens=33)
                yield put("ring 128x128/2", spread(680, 20), 3100, 272, "f32")
                yield put("ring 128x128/4", (5000, 1900), 390, 272, "f32", tokens=700)
                yield put("ring 128x256/3", spread(658, 6), 7822, 1168, "f32")


CASES = [*_dense(), *_grouped()]
