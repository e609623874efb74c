"""Linear on given 8-bit codes, and the codes: exact against integers.

acc is exact; (float)acc, the product with x_scale and the one with w_scale are each rounded to fp32,
then the result to its type: compared bit for bit with the same three roundings in numpy."""
import numpy as np
import pytest
import torch

from _util import bits_of, gpu_lib
from oracle import moe_few_oracle as MO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


def make(M, N, K, seed=0, pad_x=0, pad_w=0, lo=-128):
    g = np.random.default_rng(seed)
    xq = g.integers(lo, 128, (M, K + 16 * pad_x), dtype=np.int8)
    w = g.integers(lo, 128, (N, K + 16 * pad_w), dtype=np.int8)
    return xq, (g.random(M) * 0.05).astype(np.float32), w, (g.random(N) * 0.01).astype(np.float32)


def want(acc, xs, ws, dtype, bias=None):
    f = torch.from_numpy(acc.astype(np.float32) * xs[:, None] * ws)  # fp32 all along
    y = f.to(dtype)
    return y if bias is None else (y.float() + bias.float()).to(dtype)


def call(ql, xq, xs, w, ws, K, **kw):
    return ql.qlinear_int8(torch.from_numpy(xq).cuda()[:, :K], torch.from_numpy(xs).cuda(),
                           torch.from_numpy(w).cuda()[:, :K], torch.from_numpy(ws).cuda(), **kw)


SIZES = [(1, 512, 1024), (1, 1, 16), (2, 33, 48), (3, 5120, 272), (8, 100, 2080), (9, 31, 1040), (16, 257, 528),
         (17, 64, 2048), (32, 130, 1600), (33, 513, 144), (100, 256, 1024), (192, 300, 2064), (193, 1000, 5136),
         (400, 2056, 400), (1000, 777, 1040), (200, 17408, 272), (161, 40, 8192),
         (17, 12800, 1040), (33, 6001, 4112), (100, 2056, 8208), (1025, 33, 48), (1100, 300, 2064), (1024, 9, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_exact(ql, M, N, K, dtype):
    xq, xs, w, ws = make(M, N, K, seed=M + N, pad_x=M % 3, pad_w=N % 2)
    acc = MO.linear_codes(xq[:, :K], xs, w[:, :K], ws)[0]
    bias = torch.randn(N, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16) if M % 2 else None
    y, path = call(ql, xq, xs, w, ws, K, bias=None if bias is None else bias.cuda(), out_dtype=dtype, debug=True)
    rows = -(-M // 16) * N  # of 16 tokens
    few = M <= 16 or M <= 1024 and rows * (K + 3300) <= 24500 * min(K + 2100, 5200)
    assert path == ("int8_codes_skinny" if few else "int8_codes_tcgen05")
    assert torch.equal(y.cpu(), want(acc, xs, ws, dtype, bias))
    one = call(ql, xq, xs, w, ws[:1], K, out_dtype=dtype)
    assert torch.equal(one.cpu(), want(acc, xs, np.repeat(ws[:1], N), dtype))


def test_sums_of_one_sign_are_exact(ql):
    """Codes of -128 over a long K: every partial sum is a power of two, the last one 2^14 K."""
    for M, N, K in ((2, 40, 17408), (24, 40, 131056), (24, 1000, 131056)):
        xq, w = np.full((M, K), -128, np.int8), np.full((N, K), -128, np.int8)
        w[1] = 127
        xq[1, ::2] = 1
        one = np.ones(max(M, N), np.float32)
        y = call(ql, xq, one[:M], w, one[:N], K, out_dtype=torch.float32)
        acc = MO.linear_codes(xq, one[:M], w, one[:N])[0]
        assert np.array_equal(y.cpu().numpy(), acc.astype(np.float32))


@pytest.mark.parametrize("M", [1, 7, 16, 32, 200, 1040])
def test_output_rows_beyond_the_call_stay(ql, M):
    xq, xs, w, ws = make(M, 45, 160, seed=3)
    wide = torch.full((M + 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    y = call(ql, xq, xs, w, ws, 160, out=wide[1:M + 1, 8:53])
    acc = MO.linear_codes(xq, xs, w, ws)[0]
    assert torch.equal(y.cpu(), want(acc, xs, ws, torch.bfloat16))
    wide[1:M + 1, 8:53] = 5.0
    assert (wide == 5.0).all()


@pytest.mark.parametrize("M,K", [(1, 8), (3, 5120), (40, 264)])
def test_quantize(ql, M, K):
    g = torch.Generator().manual_seed(K)
    x = torch.randn(M, K + 8, generator=g).to(torch.bfloat16)
    x[0, :] = 0
    x[-1, 0] = 31.75  # ties: quarters of 31.75 / 127
    x[-1, 1:8] = torch.tensor([0.125, 0.375, -0.625, 31.625, -31.75, 1.125, -0.125])
    q, s = ql.quantize_int8(x.cuda()[:, :K])
    v = x[:, :K].float().numpy()
    scale = np.abs(v).max(axis=1) / np.float32(127)
    assert np.array_equal(s.cpu().numpy(), scale)
    with np.errstate(invalid="ignore", divide="ignore"):
        codes = np.where(scale[:, None] > 0, np.rint(v / scale[:, None]), 0).astype(np.int8)
    assert np.array_equal(q.cpu().numpy(), codes)


@pytest.mark.parametrize("K", [2048, 4104, 9000, 20000])
def test_quantize_ties_and_small_rows(ql, K):
    """Every mantissa as the row's largest: halves of it are ties, and for some all odd mantissas are; rows
    down to the smallest numbers."""
    g = torch.Generator().manual_seed(K)
    x = torch.randn(300, K, generator=g).clamp(-2, 2).to(torch.bfloat16)
    top = torch.arange(128, 256).repeat(3)[:300].to(torch.float32) / 64
    x[:, 5] = top.to(torch.bfloat16)
    x[:, 6::11] = (top / 2).to(torch.bfloat16)[:, None]
    x[:, 7::11] = -(top / 2).to(torch.bfloat16)[:, None]
    x[260:] = (x[260:].double() * 2.0 ** -torch.arange(90, 130)[:, None]).to(torch.bfloat16)
    q, s = ql.quantize_int8(x.cuda())
    v = x.float().numpy()
    scale = np.abs(v).max(axis=1) / np.float32(127)
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(q.cpu().numpy(), np.clip(np.rint(v / scale[:, None]), -127, 127).astype(np.int8))


def test_quantize_tells_of_nan_and_infinity(ql):
    x = torch.ones(3, 64, dtype=torch.bfloat16)
    x[0, 9], x[2, 63] = float("nan"), -float("inf")
    s = ql.quantize_int8(x.cuda())[1].cpu()
    assert s[0].isnan() and s[1] == np.float32(1) / np.float32(127) and s[2].isinf()


@pytest.mark.parametrize("M", [1, 5, 16, 30, 260, 1050])
def test_same_as_the_linear_that_quantises_itself(ql, M):
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, 1280, generator=g).to(torch.bfloat16).cuda()
    w = torch.randint(-127, 128, (300, 1280), generator=g, dtype=torch.int8).cuda()
    ws = (torch.rand(300, generator=g) * 0.01).cuda()
    bias = torch.randn(300, generator=g).to(torch.bfloat16).cuda()
    codes, scale = ql.quantize_int8(x)
    assert torch.equal(ql.qlinear_int8(codes, scale, w, ws, bias), ql.qlinear_int8_w8a8(x, w, ws, bias))


GEMM = [(20, 12000, 1040), (161, 5000, 1040), (400, 700, 4112)]  # tiles of the rest alone; whole tiles too


@pytest.mark.parametrize("M,N,K", GEMM)
def test_nothing_is_left_behind_by_waits_that_run_out(ql, M, N, K):
    """A wait limit of a few polls lets roles of the GEMM give up; the pair waits for its copies in flight
    and leaves, and the next call finds the workspace as it needs it."""
    xq, xs, w, ws = make(M, N, K, seed=6)
    args = [torch.from_numpy(a).cuda() for a in (xq, xs, w, ws)]
    space = ql.Workspace("cuda")
    whole = ql.qlinear_int8(*args, workspace=space)
    assert torch.equal(whole.cpu(), want(MO.linear_codes(xq, xs, w, ws)[0], xs, ws, torch.bfloat16))
    seen = 0
    for limit in (0, 0, 0, 1, 2, 4, 8, 16, 32, 64, 128):
        ql.set_wait_limit(limit)
        try:
            ql.qlinear_int8(*args, workspace=space)
        finally:
            ql.set_wait_limit(1 << 20)
        seen += ql.read_device_status(space.buf, clear=True)[1] & 1
        assert not space.buf[256:256 + (1 << 20)].any()
        assert torch.equal(ql.qlinear_int8(*args, workspace=space), whole)
        assert ql.read_device_status(space.buf) == (0, 0)
    assert seen


@pytest.mark.parametrize("M", [1, 12, 40, 300, 1030])
def test_graphs_and_streams(ql, M):
    sets = [[torch.from_numpy(a).cuda() for a in make(M, 600, 2064, seed=s)] for s in (1, 2)]
    alone = [ql.qlinear_int8(*a) for a in sets]
    graphs = []
    for a in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = [ql.qlinear_int8(*a), ql.qlinear_int8(*a)]
        graphs.append((g, outs))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in (0, 1, 1, 0):
        graphs[i][0].replay()
        there = ql.qlinear_int8(*sets[1 - i], stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(o, alone[i]) for o in graphs[i][1]) and torch.equal(there, alone[1 - i])


def test_refusals(ql):
    xq, xs, w, ws = [torch.from_numpy(a).cuda() for a in make(3, 32, 64)]
    y = torch.empty(3, 32, dtype=torch.bfloat16, device="cuda")
    for args, kw in [((xq.cpu(), xs, w, ws), {}), ((xq, xs.cpu(), w, ws), {}), ((xq, xs, w.cpu(), ws), {}),
                     ((xq, xs, w, ws.cpu()), {}), ((xq.to(torch.uint8), xs, w, ws), {}), ((xq, xs.double(), w, ws), {}),
                     ((xq, xs[:2], w, ws), {}), ((xq, xs, w, ws[:31]), {}), ((xq[:, :48], xs, w, ws), {}),
                     ((xq[:, :40], xs, w[:, :40], ws), {}), ((xq.t(), xs, w, ws), {}), ((xq[:0], xs[:0], w, ws), {}),
                     ((xq, xs, w, ws, y[0].float()[:32]), {}), ((xq, xs, w, ws), dict(out_dtype=torch.float64)),
                     ((xq, xs, w, ws), dict(out=y[:, :31])), ((xq, xs, w, ws), dict(out=y.int())),
                     ((xq, xs, w, ws), dict(out=y.cpu()))]:
        with pytest.raises((TypeError, ValueError, ql.QLError)):
            ql.qlinear_int8(*args, **kw)
    x = torch.randn(3, 64).to(torch.bfloat16).cuda()
    for args, kw in [((x.cpu(),), {}), ((x.float(),), {}), ((x[:, :60],), {}), ((x.t(),), {}), ((x[:0],), {}),
                     ((x,), dict(out=torch.empty(3, 48, dtype=torch.int8, device="cuda"))),
                     ((x,), dict(out_scale=torch.empty(4, device="cuda")))]:
        with pytest.raises((TypeError, ValueError, ql.QLError)):
            ql.quantize_int8(*args, **kw)
