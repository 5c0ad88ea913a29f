"""Sizes that between them take every form a product of the 8-bit operators has: rows and columns of a tile, split or
whole K, scales turned or not (fp8_gemm_form), with outputs in float32 or not and h as codes or not."""
import ctypes

from fp4_block_scaled_tensor_amd import _lib

# (rows of x, rows of the weight, k, experts; 0: one weight)
GEMM = [(17, 28672, 4096, 0), (2047, 4096, 14336, 0), (1, 70, 128, 0), (17, 70, 1100, 0), (4100, 520, 128, 0), (6144, 70, 4096, 0),
        (6144, 200, 2048, 0), (400, 520, 8191, 0), (17, 70, 2048, 0), (6144, 520, 128, 0), (8191, 1030, 128, 0),
        (4100, 70, 32768, 0), (4100, 4096, 14336, 0),
        (1, 70, 128, 3), (17, 70, 128, 3), (17, 70, 2048, 3), (8191, 200, 128, 3), (6144, 520, 128, 3), (2047, 200, 2048, 3),
        (1000, 3584, 128, 8), (6144, 70, 4096, 3), (2100, 200, 4096, 8), (6144, 1030, 128, 8), (6144, 70, 14336, 8),
        (4100, 70, 32768, 8), (6144, 1030, 14336, 32)]
GATED = [(4, 28672, 4096, 0), (8192, 28672, 4096, 0), (1, 70, 128, 0), (17, 70, 1100, 0), (4100, 520, 128, 0), (17, 70, 2048, 0),
         (6144, 70, 4096, 0), (6144, 520, 128, 0), (8191, 1030, 128, 0), (129, 2050, 32768, 0), (6144, 200, 2048, 0),
         (4100, 520, 8191, 0), (515, 200, 4096, 0), (129, 200, 300, 0),
         (1, 70, 128, 3), (17, 70, 128, 3), (17, 70, 2048, 3), (8191, 200, 128, 3), (6144, 520, 128, 3), (2047, 200, 2048, 3),
         (6144, 70, 4096, 3), (2100, 3584, 128, 8), (400, 2050, 14336, 3), (4100, 200, 128, 3), (4100, 70, 32768, 8),
         (1000, 200, 2048, 3), (6144, 1030, 14336, 32)]


def form(m, n, k, experts, gated, f32, layout=1):
    """(rows of a tile, columns, parts of K, whose scales are turned) of a product with a weight of a scale layout."""
    w = _lib.F8Operand(None, None, _lib.FP8_SCALE_E8M0, layout, n, k)
    f = (ctypes.c_int32 * 4)()
    _lib.check(_lib.load().fp8_gemm_form(m, ctypes.byref(w), experts, gated, f32, f))
    return tuple(f)


def forms(size, gated):
    """What a size takes in each of its calls: (experts, h as codes, a float32 output, rows, columns, split, turned)."""
    calls = [(1, 0), (1, 1), (2, 0), (2, 1)] if gated else [(0, 0), (0, 1)]
    out = set()
    for g, f32 in calls:
        bm, bn, parts, turned = form(*size, g, f32)
        out.add((size[3] > 0, g == 2, f32, bm, bn, parts > 1, turned))
    return out
