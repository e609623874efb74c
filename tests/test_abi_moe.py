"""Refusals of the 8-bit-code linear, the token codes and the few-token mixture-of-experts layers, before
any launch (no GPU: the addresses are fakes that are never read)."""
import ctypes

import pytest

from _util import ensure_built

V, I64, C, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(ensure_built())


HEAD = [("x", V, 16), ("M", I64, 3), ("H", I64, 64), ("ldx", I64, 64), ("logits", V, 16), ("ids", V, None),
        ("wts", V, None), ("E", C, 8), ("topk", C, 2), ("renorm", C, 0)]
TAIL = [("I", I64, 32), ("alpha", F, 1.0), ("limit", F, INF), ("ids_out", V, None), ("wts_out", V, None),
        ("h_out", V, None), ("y", V, 16), ("ldy", I64, 64), ("ws", V, 16), ("bytes", SZ, 1 << 30), ("stream", V, None)]
SPECS = {
    "quantize_int8": [("x", V, 16), ("M", I64, 3), ("K", I64, 64), ("ldx", I64, 64), ("codes", V, 16),
                      ("scale", V, 16), ("stream", V, None)],
    "qlinear_int8": [("x", V, 16), ("M", I64, 3), ("K", I64, 64), ("ldx", I64, 64), ("xs", V, 16), ("w", V, 16),
                     ("N", I64, 32), ("ldw", I64, 64), ("wsc", V, 16), ("len", I64, 32), ("bias", V, None),
                     ("out", C, 0), ("y", V, 16), ("ldy", I64, 32), ("ws", V, 16), ("bytes", SZ, 1 << 40),
                     ("stream", V, None)],
    "moe_bf16": HEAD + [("w13", V, 16), ("ld13", I64, 64), ("e13", I64, 4096), ("w2", V, 16), ("ld2", I64, 32),
                        ("e2", I64, 2048)] + TAIL,
    "moe_int8": HEAD + [("w13", V, 16), ("ld13", I64, 64), ("e13", I64, 4096), ("s13", V, 16), ("w2", V, 16),
                        ("ld2", I64, 32), ("e2", I64, 2048), ("s2", V, 16)] + TAIL,
    "moe_int4": HEAD + [("w13", V, 16), ("ld13", I64, 32), ("e13", I64, 2048), ("s13", V, 16), ("lds13", I64, 2),
                        ("es13", I64, 128), ("z13", V, 16), ("ldz13", I64, 2), ("ez13", I64, 128), ("w2", V, 16),
                        ("ld2", I64, 16), ("e2", I64, 1024), ("s2", V, 16), ("lds2", I64, 1), ("es2", I64, 64),
                        ("z2", V, 16), ("ldz2", I64, 1), ("ez2", I64, 64), ("fmt", C, 0), ("group", I64, 32)] + TAIL,
}
MOE = [(dict(x=None), INVALID), (dict(w13=None), INVALID), (dict(w2=None), INVALID), (dict(y=None), INVALID),
       (dict(M=0), INVALID), (dict(M=-1), INVALID), (dict(H=0), INVALID), (dict(I=0), INVALID), (dict(E=0), INVALID),
       (dict(topk=0), INVALID), (dict(ldx=56), INVALID), (dict(ldy=63), INVALID), (dict(logits=None), INVALID),
       (dict(ids=16, wts=16), INVALID), (dict(logits=None, ids=16), INVALID), (dict(alpha=NAN), INVALID),
       (dict(alpha=INF), INVALID), (dict(limit=-1.0), INVALID), (dict(limit=NAN), INVALID), (dict(ld13=16), INVALID),
       (dict(e13=-16), INVALID), (dict(M=65), UNSUPPORTED), (dict(topk=9), UNSUPPORTED),
       (dict(topk=17, E=32), UNSUPPORTED), (dict(E=1025), UNSUPPORTED), (dict(H=32800, ldx=32800, ldy=32800), UNSUPPORTED),
       (dict(x=24), ALIGNMENT), (dict(w13=8), ALIGNMENT), (dict(w2=8), ALIGNMENT), (dict(ldx=68), ALIGNMENT),
       (dict(e13=4100), ALIGNMENT), (dict(y=17), ALIGNMENT), (dict(logits=17), ALIGNMENT), (dict(ws=None), WORKSPACE),
       (dict(bytes=4096), WORKSPACE), (dict(ws=8), ALIGNMENT)]
CASES = ([(n, *c) for n in ("moe_bf16", "moe_int8", "moe_int4") for c in MOE]
         + [("moe_bf16", dict(H=60, ldx=64), UNSUPPORTED), ("moe_int8", dict(H=56, ldx=64), UNSUPPORTED),
            ("moe_int4", dict(H=48, ldx=64, lds13=4, ldz13=4), UNSUPPORTED), ("moe_int8", dict(s13=None), INVALID),
            ("moe_int8", dict(s2=None), INVALID), ("moe_int8", dict(s13=18), ALIGNMENT),
            ("moe_int4", dict(s13=None), INVALID), ("moe_int4", dict(fmt=2), INVALID),
            ("moe_int4", dict(lds13=1), INVALID), ("moe_int4", dict(ldz13=1), INVALID),
            ("moe_int4", dict(es13=-1), INVALID), ("moe_int4", dict(group=0), INVALID),
            ("moe_int4", dict(group=48, lds13=4), UNSUPPORTED), ("moe_int4", dict(group=16, lds13=4, ldz13=4, lds2=2, ldz2=2), UNSUPPORTED),
            ("moe_int4", dict(s2=17), ALIGNMENT)]
         + [("qlinear_int8", *c) for c in [
             (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(w=None), INVALID), (dict(wsc=None), INVALID),
             (dict(y=None), INVALID), (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
             (dict(ldx=48), INVALID), (dict(ldw=48), INVALID), (dict(ldy=31), INVALID), (dict(len=2), INVALID),
             (dict(out=3), INVALID), (dict(out=-1), INVALID), (dict(K=56), UNSUPPORTED), (dict(M=(1 << 22) + 1), UNSUPPORTED),
             (dict(N=(1 << 24) + 1, ldy=1 << 25, len=1), UNSUPPORTED),
             (dict(K=131072, ldx=131072, ldw=131072), UNSUPPORTED), (dict(x=8), ALIGNMENT), (dict(w=8), ALIGNMENT),
             (dict(ldx=72), ALIGNMENT), (dict(ldw=72), ALIGNMENT), (dict(xs=18), ALIGNMENT), (dict(y=17), ALIGNMENT),
             (dict(y=18, out=2), ALIGNMENT), (dict(bias=17), ALIGNMENT), (dict(ws=None), WORKSPACE),
             (dict(bytes=1 << 20), WORKSPACE), (dict(M=100, bytes=1 << 21), WORKSPACE), (dict(ws=8), ALIGNMENT)]]
         + [("quantize_int8", *c) for c in [
             (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scale=None), INVALID), (dict(M=0), INVALID),
             (dict(K=0), INVALID), (dict(ldx=56), INVALID), (dict(K=60), UNSUPPORTED), (dict(x=8), ALIGNMENT),
             (dict(codes=8), ALIGNMENT), (dict(scale=18), ALIGNMENT), (dict(ldx=68), ALIGNMENT)]])


@pytest.mark.parametrize("name,change,want", CASES, ids=[f"{n}-{'-'.join(f'{k}={v}' for k, v in c.items())}"
                                                         for n, c, _ in CASES])
def test_refused_before_launch(lib, name, change, want):
    spec = SPECS[name]
    f = getattr(lib, name)
    f.restype = C
    path = C(-1)
    last = [] if name == "quantize_int8" else [ctypes.byref(path)]
    f.argtypes = [t for _, t, _ in spec] + [ctypes.POINTER(C)] * len(last)
    assert f(*[change.get(k, d) for k, _, d in spec], *last) == want
    if last:
        assert path.value == 0


def test_workspaces(lib):
    f = lib.ql_workspace_bytes
    f.restype = SZ
    f.argtypes = [C, I64, I64, I64, C, C]
    base = 256 + (1 << 20)
    assert f(9, 1, 64, 64, 0, 0) > base and f(9, 4096, 17408, 5120, 0, 0) >= base + 4096 * 5120 * 2
    assert f(10, 64, 4096, 2048, 256, 16) >= base + 64 * 16 * 2048 * 2
    for op in (9, 10):  # sizes that the calls refuse: an answer all the same
        for M, N, K in ((0, 8, 8), (1 << 40, 8, 8), (8, 1 << 40, 8), (8, 8, 1 << 40)):
            assert f(op, M, N, K, 8, 2) >= base
    assert f(10, 1, 64, 64, 0, 2) == 0 and f(9, -1, 8, 8, 0, 0) == 0
