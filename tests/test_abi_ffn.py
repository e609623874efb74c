"""Refusals of the 4-bit linear and the gated block's entry points, before any launch (no GPU: the
addresses are fakes that are never read)."""
import ctypes

import pytest

from _util import ensure_built

V, I64, C, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(ensure_built())


SPECS = {
    "qlinear_int4": [("x", V, 16), ("M", I64, 1), ("K", I64, 256), ("ldx", I64, 256), ("w", V, 16), ("N", I64, 64),
                     ("ldw", I64, 128), ("s", V, 16), ("fmt", C, 0), ("lds", I64, 2), ("z", V, 16), ("ldz", I64, 2),
                     ("group", I64, 128), ("bias", V, None), ("y", V, 16), ("ldy", I64, 64), ("stream", V, None)],
    "gated_ffn_int4": [("x", V, 16), ("M", I64, 1), ("K", I64, 256), ("ldx", I64, 256), ("w", V, 16), ("N", I64, 64),
                       ("ldw", I64, 128), ("s", V, 16), ("fmt", C, 0), ("lds", I64, 2), ("z", V, 16), ("ldz", I64, 2),
                       ("group", I64, 128), ("alpha", F, 1.0), ("limit", F, INF), ("y", V, 16), ("ldy", I64, 64),
                       ("stream", V, None)],
    "gated_ffn": [("x", V, 16), ("M", I64, 1), ("H", I64, 64), ("ldx", I64, 64), ("w", V, 16), ("I", I64, 64),
                  ("ldw", I64, 64), ("alpha", F, 1.0), ("limit", F, INF), ("h", V, 16), ("ldh", I64, 64),
                  ("save", C, 2), ("ckpt", V, 16), ("scale", V, 16), ("ws", V, 16), ("bytes", SZ, 1 << 30),
                  ("stream", V, None)],
    "gated_ffn_backward": [("dh", V, 16), ("ld_dh", I64, 64), ("x", V, 16), ("M", I64, 1), ("H", I64, 64),
                           ("ldx", I64, 64), ("w", V, 16), ("I", I64, 64), ("ldw", I64, 64), ("alpha", F, 1.0),
                           ("limit", F, INF), ("save", C, 2), ("ckpt", V, 16), ("scale", V, 16), ("dx", V, 16),
                           ("ld_dx", I64, 64), ("dw", V, 16), ("ld_dw", I64, 64), ("ws", V, 16),
                           ("bytes", SZ, 1 << 30), ("stream", V, None)],
}

INT4 = [(dict(x=None), INVALID), (dict(w=None), INVALID), (dict(s=None), INVALID), (dict(y=None), INVALID),
        (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(M=-3), INVALID),
        (dict(ldx=248), INVALID), (dict(ldw=112), INVALID), (dict(ldy=63), INVALID), (dict(lds=1), INVALID),
        (dict(ldz=1), INVALID), (dict(group=0), INVALID), (dict(fmt=2), INVALID),
        (dict(M=65536), UNSUPPORTED), (dict(K=240, lds=9), UNSUPPORTED), (dict(group=96, lds=9, ldz=9), UNSUPPORTED),
        (dict(group=16, lds=16, ldz=16), UNSUPPORTED), (dict(x=24), ALIGNMENT), (dict(w=8), ALIGNMENT),
        (dict(s=17), ALIGNMENT), (dict(ldx=260), ALIGNMENT), (dict(ldw=136), ALIGNMENT)]
ACT = [(dict(alpha=NAN), INVALID), (dict(alpha=INF), INVALID), (dict(limit=-1.0), INVALID), (dict(limit=NAN), INVALID)]
FFN = [(dict(M=0), INVALID), (dict(H=0), INVALID), (dict(I=0), INVALID), (dict(ldx=56), INVALID),
       (dict(ldw=56), INVALID), (dict(H=60), UNSUPPORTED), (dict(I=60), UNSUPPORTED), (dict(M=(1 << 22) + 1), UNSUPPORTED),
       (dict(ldx=68), ALIGNMENT), (dict(ldw=68), ALIGNMENT), (dict(x=8), ALIGNMENT), (dict(w=8), ALIGNMENT),
       (dict(ckpt=8), ALIGNMENT), (dict(ws=None), WORKSPACE), (dict(bytes=1024), WORKSPACE), (dict(ws=8), ALIGNMENT),
       (dict(ckpt=None), INVALID), (dict(scale=None), INVALID), (dict(save=3), INVALID)]
CASES = ([("qlinear_int4", *c) for c in INT4] + [("gated_ffn_int4", *c) for c in INT4 + ACT]
         + [("gated_ffn", *c) for c in FFN + ACT + [(dict(x=None), INVALID), (dict(w=None), INVALID),
                                                    (dict(h=None), INVALID), (dict(ldh=56), INVALID),
                                                    (dict(ldh=68), ALIGNMENT), (dict(h=8), ALIGNMENT)]]
         + [("gated_ffn_backward", *c) for c in FFN + ACT + [
             (dict(dh=None), INVALID), (dict(dx=None, dw=None), INVALID), (dict(x=None), INVALID),
             (dict(w=None), INVALID), (dict(save=0), INVALID), (dict(ld_dh=56), INVALID), (dict(ld_dx=56), INVALID),
             (dict(ld_dw=56), INVALID), (dict(ld_dh=68), ALIGNMENT), (dict(ld_dx=68), ALIGNMENT),
             (dict(ld_dw=68), ALIGNMENT), (dict(dh=8), ALIGNMENT), (dict(dx=8), ALIGNMENT), (dict(dw=8), ALIGNMENT)]]
         + [("qlinear_int4", dict(y=17), ALIGNMENT), ("qlinear_int4", dict(bias=17), ALIGNMENT),
            ("gated_ffn_int4", dict(y=17), ALIGNMENT), ("gated_ffn", dict(scale=18), ALIGNMENT),
            ("gated_ffn_backward", dict(scale=18), ALIGNMENT)])


@pytest.mark.parametrize("name,change,want", CASES, ids=[f"{n}-{'-'.join(f'{k}={v}' for k, v in c.items())}"
                                                         for n, c, _ in CASES])
def test_refused_before_launch(lib, name, change, want):
    spec = SPECS[name]
    f = getattr(lib, name)
    f.restype = C
    f.argtypes = [t for _, t, _ in spec] + [ctypes.POINTER(C)]
    path = C(-1)
    assert f(*[change.get(k, d) for k, _, d in spec], ctypes.byref(path)) == want
    assert path.value == 0


def test_workspace_of_the_gated_block(lib):
    f = lib.ql_workspace_bytes
    f.restype = SZ
    f.argtypes = [C, I64, I64, I64, C, C]
    assert f(7, 4096, 17408, 5120, 0, 0) >= f(7, 1, 8, 8, 0, 0) >= 256 + (1 << 20)
    assert f(8, 4096, 17408, 5120, 0, 0) >= 256 + (1 << 20) + 4096 * 2 * 17408 * 2
    assert f(8, -1, 8, 8, 0, 0) == 0
    for op in (7, 8):  # sizes that the calls refuse: an answer all the same
        for M, N, K in ((0, 8, 8), (8, 0, 8), (8, 8, 0), (0, 0, 0), (1 << 40, 8, 8), (8, 1 << 40, 1 << 40)):
            assert f(op, M, N, K, 0, 0) >= 256 + (1 << 20)
