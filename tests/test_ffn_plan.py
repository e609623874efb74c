"""How the gated block's GEMMs are laid out (ql_gated_ffn_plan; no GPU): its answers hold together,
and the shapes that the GPU tests of cut tiles use are cut as those tests need."""
import ctypes

import pytest

from _util import ensure_built

I64, I32 = ctypes.c_int64, ctypes.c_int32
FWD, DX, DW = 0, 1, 2
NONE, BF16, INT8 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(ensure_built())
    lib.ql_gated_ffn_plan.restype = ctypes.c_int
    lib.ql_gated_ffn_plan.argtypes = [ctypes.c_int, I64, I64, I64, ctypes.c_int, ctypes.POINTER(I32)]
    lib.ql_workspace_bytes.restype = ctypes.c_size_t
    lib.ql_workspace_bytes.argtypes = [ctypes.c_int, I64, I64, I64, ctypes.c_int, ctypes.c_int]
    return lib


def plan(lib, gemm, M, I, H, mode):
    out = (I32 * 6)()
    assert lib.ql_gated_ffn_plan(gemm, M, I, H, mode, out) == 0
    return dict(zip(("pairs", "width", "whole", "cut", "parts", "launches"), out))


# (GEMM, mode, M, H, I, whole tiles before the cut ones, launches of the call's GEMMs)
CUT = [(FWD, BF16, 40, 4096, 72, False, 1), (FWD, INT8, 40, 4096, 72, False, 1),
       (FWD, NONE, 4104, 4096, 520, True, 1), (FWD, BF16, 4104, 4096, 520, True, 1), (FWD, INT8, 4104, 4096, 520, True, 1),
       (FWD, INT8, 268, 3472, 5104, True, 1), (FWD, NONE, 4962, 2304, 24, False, 1),
       (DX, 1, 2406, 8, 1136, False, 1), (DW, 1, 2406, 8, 1136, False, 1), (DX, 1, 1, 6176, 1968, True, 1),
       (DW, 1, 2311, 8, 4800, True, 1), (DX, 1, 5645, 8, 7440, False, 2), (DX, 1, 6899, 784, 2352, True, 2),
       (DX, 1, 8439, 568, 6952, True, 2), (DW, 1, 8439, 568, 6952, True, 2), (DW, 0, 3020, 296, 5288, True, 1),
       (DX, 0, 40, 2056, 2448, False, 1)]


@pytest.mark.parametrize("gemm,mode,M,H,I,whole,launches", CUT)
def test_shapes_that_are_cut(lib, gemm, mode, M, H, I, whole, launches):
    p = plan(lib, gemm, M, I, H, mode)
    assert p["cut"] > 0 and p["parts"] > 1 and (p["whole"] > 0) == whole and p["launches"] == launches
    assert p["cut"] * p["parts"] <= p["pairs"]


def test_one_gradient_alone_is_cut_otherwise(lib):
    both, alone = plan(lib, DX, 40, 2448, 2056, 1), plan(lib, DX, 40, 2448, 2056, 0)
    assert (both["cut"], both["parts"]) != (alone["cut"], alone["parts"])


@pytest.mark.parametrize("M,H,I", [(1, 8, 8), (17, 5120, 17408), (333, 1024, 2040), (2048, 4096, 2048),
                                   (4096, 5120, 17408), (1 << 22, 8, 8), (8, 1 << 20, 1 << 20)])
def test_tiles_cover_the_output_and_parts_fit_the_workspace(lib, M, H, I):
    part = 2 * 256 * 128 * 4  # a part's sums of both CTAs
    for gemm, modes in ((FWD, (NONE, BF16, INT8)), (DX, (0, 1)), (DW, (0, 1))):
        slots = []
        for mode in modes:
            p = plan(lib, gemm, M, I, H, mode)
            if p["pairs"] == 0:
                assert gemm == FWD and mode == NONE and (p["width"], p["cut"], p["launches"]) == (0, 0, 1)
                continue
            rows, cols = {FWD: (M, I), DX: (M, H), DW: (2 * I, H)}[gemm]
            outs = p["width"] // 2 if gemm == FWD else p["width"]
            assert p["whole"] + p["cut"] == -(-rows // 256) * -(-cols // outs)
            assert p["width"] % 32 == 0 and 64 <= p["width"] <= 256 and 1 <= p["pairs"] <= 76
            slots.append(p["cut"] * p["parts"] * part)
        op, extra = (7, 0) if gemm == FWD else (8, M * 2 * I * 2)
        assert lib.ql_workspace_bytes(op, M, I, H, 0, 0) >= 256 + (1 << 20) + extra + max(slots + [0])


def test_refusals(lib):
    out = (I32 * 6)()
    f = lib.ql_gated_ffn_plan
    assert f(FWD, 8, 64, 64, NONE, None) == 1
    for bad in ((3, 8, 64, 64, 0), (-1, 8, 64, 64, 0), (FWD, 8, 64, 64, 3), (DX, 8, 64, 64, 2), (FWD, 0, 64, 64, 0)):
        assert f(*bad, out) == 1
    assert f(FWD, 8, 60, 64, 0, out) == 2
