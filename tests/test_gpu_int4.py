"""4-bit group-scaled linear and the gated block on such weights, against the 64-bit definition.

Tolerances.  Every product x (q - z) is exact in fp32; each of the K additions of a sum rounds or
truncates by at most 2^-23 of the sum of magnitudes, so |sum - exact| <= K 2^-23 sum|x w|; the
result is rounded to bf16 (1 ulp)."""
import numpy as np
import pytest
import torch

from _util import bits_of, gpu_lib
from oracle import ffn_oracle as O
from oracle import formats as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


def make(M, N, K, group, zeros=True, dtype=torch.bfloat16, seed=0, pad_w=0, pad_x=0, pad_s=0):
    g = torch.Generator().manual_seed(seed)
    groups = -(-K // group)
    ld = -(-K // 32) * 16 + 16 * pad_w
    w = torch.randint(0, 256, (N, ld), generator=g, dtype=torch.uint8)
    s = ((torch.rand(N, groups + pad_s, generator=g) + 0.1) * 0.02).to(dtype)
    s[:, groups:] = float("nan")  # never read
    z = torch.randint(0, 16, (N, groups + pad_s), generator=g, dtype=torch.uint8) if zeros else None
    x = torch.randn(M, K + 8 * pad_x, generator=g).to(torch.bfloat16)
    x[:, K:] = float("nan")
    return x.cuda()[:, :K], w.cuda(), s.cuda(), None if z is None else z.cuda()


def reference(x, w, s, z, K, group):
    wd = O.int4_dequant(w.cpu().numpy(), s.double().cpu().numpy(), None if z is None else z.cpu().numpy(), K, group)
    return O.linear(x.double().cpu().numpy(), wd)


def check(y, ref, absum, K):
    got = F.bf16_to_f64(bits_of(y))
    tol = K * 2.0 ** -23 * absum + F.bf16_ulp(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist())


@pytest.mark.parametrize("group", [32, 64, 128, 256, 1 << 20])
@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (1, 1, 32), (2, 17, 96), (7, 33, 416), (8, 31, 128), (9, 48, 1184),
                                   (16, 65, 2080), (17, 130, 544), (32, 64, 1024), (33, 100, 288), (70, 19, 160)])
def test_int4_matches_the_definition(ql, M, N, K, group):
    dtype, zeros = ((torch.bfloat16, True), (torch.float16, False))[(M + group // 32) % 2]
    x, w, s, z = make(M, N, K, group, zeros, dtype, seed=M * 1000 + N)
    y, path = ql.qlinear_int4(x, w, s, z, group=group, debug=True)
    assert path == "int4_skinny"
    check(y, *reference(x, w, s, z, K, group), K)


def sampled(N, n=60):
    return np.unique(np.concatenate([[0, 1, N // 2, N - 2, N - 1], np.random.default_rng(N).integers(0, N, n)]))


# K shares over clusters of CTAs, one token's activations staged in several pieces, more tokens' in
# the rings, rows for two CTAs per SM and more: every token, sampled rows
@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (128, True), (512, False)])
@pytest.mark.parametrize("M,N,K", [(1, 5000, 17408), (3, 5000, 17408), (4, 5000, 17376), (4, 96, 17408), (8, 640, 8224),
                                   (16, 640, 8224), (24, 330, 4128), (2, 19500, 3232), (4, 19500, 3232)])
def test_int4_large_sampled(ql, M, N, K, group, zeros):
    x, w, s, z = make(M, N, K, group, zeros, torch.bfloat16, seed=N + M)
    y = ql.qlinear_int4(x, w, s, z, group=group)
    rows = torch.from_numpy(sampled(N)).cuda()
    ref, absum = reference(x, w[rows], s[rows], None if z is None else z[rows], K, group)
    check(y[:, rows].contiguous(), ref, absum, K)


# each number of warps, tokens and rows that the launch chooses between: up to a row tile per SM (4864
# rows), from four per SM on (19456), K of fewer blocks than warps and of more
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("M", [1, 2, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("N,K", [(4864, 4000), (4865, 4000), (19457, 672), (200, 17408), (100, 3968)])
def test_int4_every_variant_sampled(ql, M, N, K, group, zeros):
    x, w, s, z = make(M, N, K, group, zeros, torch.bfloat16, seed=N + K + M)
    y = ql.qlinear_int4(x, w, s, z, group=group)
    rows = torch.from_numpy(sampled(N, 24)).cuda()
    ref, absum = reference(x, w[rows], s[rows], None if z is None else z[rows], K, group)
    check(y[:, rows].contiguous(), ref, absum, K)


def test_int4_infinite_scale_of_a_short_last_block(ql):
    """K ends inside a block of 128: the groups after its end do not exist, whatever the last one's
    scale is; a row with an infinite scale is infinite where its group's sum is not zero."""
    M, N, K, group = 2, 20, 160, 32
    x, w, s, z = make(M, N, K, group, True, torch.bfloat16, seed=5)
    s[3, 4] = float("inf")
    y = ql.qlinear_int4(x, w, s, z, group=group)
    wd = O.int4_dequant(w.cpu().numpy(), np.ones((N, 5)), z.cpu().numpy(), K, group)
    last = (x.double().cpu().numpy()[:, 128:] * wd[3, 128:]).sum(1)
    assert np.all(last != 0)
    assert np.array_equal(y[:, 3].double().cpu().numpy(), np.sign(last) * np.inf)


@pytest.mark.parametrize("group,zeros", [(64, True), (128, False)])
@pytest.mark.parametrize("M,I,H", [(1, 9750, 3232), (4, 9750, 3232), (3, 1030, 8224), (12, 1030, 8224)])
def test_gated_int4_large_sampled(ql, M, I, H, group, zeros):
    x, w, s, z = make(M, 2 * I, H, group, zeros, torch.float16, seed=I + M)
    h = ql.gated_ffn_int4(x, w, s, z, group=group)
    o = sampled(I)
    rows = torch.from_numpy(np.concatenate([o, I + o])).cuda()
    gu, absum = reference(x, w[rows], s[rows], None if z is None else z[rows], H, group)
    n = len(o)
    g, u, G, U = gu[:, :n], gu[:, n:], absum[:, :n], absum[:, n:]
    got = F.bf16_to_f64(bits_of(h[:, torch.from_numpy(o).cuda()].contiguous()))
    assert np.all(np.abs(got - O.gated(g, u)) <= h_tol(g, u, G, U, H, 1.0, np.inf))


@pytest.mark.parametrize("group", [32, 128])
def test_int4_strides_bias_and_guard_columns(ql, group):
    M, N, K = 5, 70, 352
    x, w, s, z = make(M, N, K, group, seed=1, pad_w=3, pad_x=2, pad_s=5)
    bias = torch.randn(N).to(torch.bfloat16).cuda()
    wide = torch.full((M, N + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    ql.qlinear_int4(x, w, s, z, bias, group=group, out=wide[:, 4:4 + N])
    ref, absum = reference(x, w, s, z, K, group)
    got = F.bf16_to_f64(bits_of(wide[:, 4:4 + N].contiguous()))
    b = bias.double().cpu().numpy()
    # the sum is rounded to bf16, the bias added and the result rounded again
    tol = K * 2.0 ** -23 * absum + F.bf16_ulp(ref) + F.bf16_ulp(np.abs(ref) + np.abs(b))
    assert np.all(np.abs(got - (ref + b)) <= tol)
    assert torch.all(wide[:, :4] == 7.0) and torch.all(wide[:, 4 + N:] == 7.0)


def test_int4_extreme_zero_points_and_scales(ql):
    """Zero points 0 and 127, a zero scale, and fp16's smallest subnormal as a scale."""
    M, N, K, group = 2, 16, 256, 64
    x, w, s, z = make(M, N, K, group, True, torch.float16, seed=2)
    z[0], z[1] = 0, 127
    s[2], s[3] = 0.0, 2.0 ** -24
    y = ql.qlinear_int4(x, w, s, z, group=group)
    check(y, *reference(x, w, s, z, K, group), K)
    assert torch.all(y[:, 2] == 0)


def test_int4_tokens_do_not_touch_each_other(ql):
    """A token of infinities or NaNs changes its own outputs only; the others keep their bits."""
    x, w, s, z = make(4, 40, 256, 128, seed=3)
    y = ql.qlinear_int4(x, w, s, z)
    x2 = x.clone()
    x2[1, 5], x2[2, 7] = float("nan"), float("inf")
    y2 = ql.qlinear_int4(x2, w, s, z)
    assert torch.equal(y2[0], y[0]) and torch.equal(y2[3], y[3])
    assert torch.all(torch.isnan(y2[1])) and not torch.any(torch.isfinite(y2[2]))


def test_int4_row_offsets_past_32_bits(ql):
    N, K, ld = 66000, 64, 65552  # the last rows start beyond 2^32 bytes
    w = torch.zeros(N, ld, dtype=torch.uint8, device="cuda")
    w[-3:, :32] = torch.randint(0, 256, (3, 32), dtype=torch.uint8, device="cuda")
    s = torch.full((N, 1), 0.5, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(1, K, device="cuda").to(torch.bfloat16)
    y = ql.qlinear_int4(x, w, s, group=64)
    check(y[:, -3:].contiguous(), *reference(x, w[-3:, :32].contiguous(), s[-3:], None, K, 64), K)


def test_int4_other_stream_and_graph(ql):
    x, w, s, z = make(3, 96, 640, 128, seed=4)
    want = ql.qlinear_int4(x, w, s, z)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = ql.qlinear_int4(x, w, s, z, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ql.qlinear_int4(x, w, s, z, out=out)
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ql.qlinear_int4(x, w, s, z))


def test_int4_python_refusals(ql):
    x, w, s, z = make(2, 32, 256, 128)
    for bad in (dict(w=w.to(torch.int8)), dict(w_scale=s.float()), dict(w_zero=z.int()), dict(x=x.float()),
                dict(bias=torch.zeros(32, device="cuda")), dict(w=w.cpu()), dict(w_scale=s.cpu()),
                dict(w_zero=z.cpu()), dict(bias=torch.zeros(32, dtype=torch.bfloat16)),
                dict(out=torch.empty(2, 32, dtype=torch.bfloat16))):
        with pytest.raises(TypeError):
            ql.qlinear_int4(**{**dict(x=x, w=w, w_scale=s, w_zero=z), **bad})
    for bad in (dict(w=w[:, :64]), dict(w_scale=s[:, :1]), dict(w_zero=z[:, :1]), dict(w_scale=s[:16]), dict(group=0)):
        with pytest.raises(ValueError):
            ql.qlinear_int4(**{**dict(x=x, w=w, w_scale=s, w_zero=z), **bad})
    with pytest.raises(ValueError):
        ql.gated_ffn_int4(x, w[:31], s[:31], z[:31])
    with pytest.raises(ql.QLError) as e:
        ql.qlinear_int4(x[:, :240], w, s.repeat(1, 4), group=48)
    assert e.value.status == 2


# ------------------------------------------------------------------------------- gated block
def h_tol(g, u, G, U, K, alpha, limit):
    """|g - exact| <= K 2^-23 G carried through silu(a g') u' (|silu'| <= 1.1, clamps are
    1-Lipschitz), 2^-17 |h| for the fast exponential and quotient, and the bf16 rounding."""
    dg, du = K * 2.0 ** -23 * G, K * 2.0 ** -23 * U
    uc, act = np.clip(u, -limit, limit), O.silu(alpha * np.minimum(g, limit))
    h = act * uc
    return 1.1 * abs(alpha) * (np.abs(uc) + du) * dg + np.abs(act) * du + 2.0 ** -17 * np.abs(h) + F.bf16_ulp(h)


@pytest.mark.parametrize("alpha,limit", [(1.0, None), (1.5, 0.7)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,I,H", [(1, 1, 32), (1, 100, 1024), (5, 33, 416), (8, 16, 128), (13, 47, 1184),
                                   (32, 64, 544), (40, 17, 288)])
def test_gated_int4_matches_the_definition(ql, M, I, H, group, alpha, limit):
    x, w, s, z = make(M, 2 * I, H, group, M % 2 == 1, torch.float16 if I % 2 else torch.bfloat16, seed=I)
    h, path = ql.gated_ffn_int4(x, w, s, z, group=group, swiglu_alpha=alpha, swiglu_limit=limit, debug=True)
    assert path == "gated_ffn_int4"
    gu, absum = reference(x, w, s, z, H, group)
    g, u, G, U = gu[:, :I], gu[:, I:], absum[:, :I], absum[:, I:]
    lim = np.inf if limit is None else limit
    got = F.bf16_to_f64(bits_of(h))
    assert np.all(np.abs(got - O.gated(g, u, alpha, lim)) <= h_tol(g, u, G, U, H, alpha, lim))


def test_gated_int4_non_finite_tokens(ql):
    x, w, s, z = make(4, 2 * 24, 256, 128, seed=6)
    h = ql.gated_ffn_int4(x, w, s, z, swiglu_limit=2.0)
    x2 = x.clone()
    x2[2, 9] = float("nan")
    h2 = ql.gated_ffn_int4(x2, w, s, z, swiglu_limit=2.0)
    assert torch.equal(h2[[0, 1, 3]], h[[0, 1, 3]]) and torch.all(torch.isnan(h2[2]))
