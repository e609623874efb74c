"""The gated feed-forward block on bf16 weights: forward, checkpoints and backward pass against the
64-bit definition.

Tolerances, derived from the arithmetic:
  sums       bf16 products are exact in fp32; each of the K additions rounds or truncates by at most
             2^-23 of the sum of magnitudes: K 2^-23 sum|x w|
  activation 2^-17 relative (fast exponential and quotient), carried through |silu'| <= 1.1
  int8       half a step and the error of the value itself; the scale is amax / 127 in fp32
  backward   from the checkpoint that the forward returned: dg, du are rounded to bf16 (2^-8) before
             their products, whose sums are bounded as above
  outputs    1 bf16 ulp"""
import numpy as np
import pytest
import torch

from _util import bits_of, gpu_lib
from oracle import ffn_oracle as O
from oracle import formats as F

pytestmark = pytest.mark.gpu

E = 2.0 ** -23


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


def make(M, H, I, seed=0, pad=0, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, H + 8 * pad, generator=g).to(torch.bfloat16)
    w = (gain * torch.randn(2 * I, H + 8 * pad, generator=g) / H ** 0.5).to(torch.bfloat16)
    dh = torch.randn(M, I + 8 * pad, generator=g).to(torch.bfloat16)
    for t, n in ((x, H), (w, H), (dh, I)):
        t[:, n:] = float("nan")  # never read
    return x.cuda()[:, :H], w.cuda()[:, :H], dh.cuda()[:, :I]


def f64(t):
    return t.double().cpu().numpy()


def forward_reference(x, w, I):
    gu, absum = O.linear(f64(x), f64(w))
    return gu[:, :I], gu[:, I:], absum[:, :I], absum[:, I:]


def check_h(h, g, u, G, U, K, alpha=1.0, limit=np.inf):
    uc, act = np.clip(u, -limit, limit), O.silu(alpha * np.minimum(g, limit))
    dg, du = K * E * G, K * E * U
    ref = act * uc
    tol = 1.1 * abs(alpha) * (np.abs(uc) + du) * dg + np.abs(act) * du + 2.0 ** -17 * np.abs(ref) + F.bf16_ulp(ref)
    bad = ~(np.abs(F.bf16_to_f64(bits_of(h.contiguous())) - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist())


def kept(saved, I):
    """The checkpoint's values of g and u as the kernel forms them (code * scale in fp32)."""
    d = saved.data[:, :, :I].float().cpu().numpy()
    if saved.mode == "int8":
        d = d * np.repeat(saved.scale.cpu().numpy(), 128, axis=2)[:, :, :I]
    return d[:, 0].astype(np.float64), d[:, 1].astype(np.float64)


def check_backward(dx, dw, dh, x, w, g, u, alpha=1.0, limit=np.inf):
    dh, x, w = f64(dh), f64(x), f64(w)
    rdx, rdw, dgu = O.backward(dh, x, w, g, u, alpha, limit)
    t = alpha * np.minimum(g, limit)
    s = O.sigmoid(t)
    mag_g = np.abs(dh * np.clip(u, -limit, limit) * alpha) * (s + np.abs(t) * s)
    mag_u = np.abs(dh * t) * s
    err = 2.0 ** -8 * np.abs(dgu) + 2.0 ** -17 * np.concatenate([mag_g, mag_u], axis=1)
    for got, ref, e, a, b, K in ((dx, rdx, err, np.abs(dgu), np.abs(w), w.shape[0]),
                                 (dw, rdw, err.T, np.abs(dgu).T, np.abs(x), x.shape[0])):
        if got is None:
            continue
        tol = (e + K * E * (a + e)) @ b + F.bf16_ulp(ref)
        bad = ~(np.abs(F.bf16_to_f64(bits_of(got.contiguous())) - ref) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist())


SHAPES = [(1, 8, 8), (1, 512, 264), (3, 72, 40), (13, 264, 72), (32, 1024, 136), (33, 128, 128), (127, 64, 8),
          (128, 320, 200), (129, 8, 256), (256, 512, 128), (257, 1000, 520), (700, 264, 1032)]


@pytest.mark.parametrize("M,H,I", SHAPES + [(16, 40, 9736), (17, 40, 9736), (32, 40, 9728), (33, 72, 2432), (33, 72, 2440), (40, 2056, 2448), (300, 328, 488),
                                         (1000, 136, 152), (2400, 64, 72), (257, 320, 1000)])
def test_forward(ql, M, H, I):
    x, w, _ = make(M, H, I, seed=M)
    h, path = ql.gated_ffn(x, w, debug=True)
    few = M <= 16 or -(-M // 32) * -(-I // 16) <= (608 if M <= 32 else 304)
    assert path == ("gated_ffn_skinny" if few else "gated_ffn_tcgen05")
    check_h(h, *forward_reference(x, w, I), H)


# each number of warps and CTAs that a few tokens' launch chooses between: up to a CTA of 16 outputs
# per SM (2432) and more, K of few blocks and of many
@pytest.mark.parametrize("M", [1, 7, 9, 16, 17, 32])
@pytest.mark.parametrize("H,I", [(2016, 2432), (2024, 2432), (2024, 2440), (8200, 80), (520, 5000)])
def test_few_tokens_every_variant_sampled(ql, M, H, I):
    x, w, _ = make(M, H, I, seed=H + I + M)
    h = ql.gated_ffn(x, w)
    o = np.unique(np.concatenate([[0, 1, I // 2, I - 1], np.random.default_rng(I).integers(0, I, 40)]))
    rows = torch.from_numpy(np.concatenate([o, I + o])).cuda()
    check_h(h[:, torch.from_numpy(o).cuda()], *forward_reference(x, w[rows], len(o)), H)


@pytest.mark.parametrize("save", ["bf16", "int8"])
@pytest.mark.parametrize("M,H,I", SHAPES)
def test_checkpoint_and_backward(ql, M, H, I, save):
    x, w, dh = make(M, H, I, seed=M + 1)
    h, saved, path = ql.gated_ffn(x, w, save=save, debug=True)
    assert path == "gated_ffn_tcgen05"
    g, u, G, U = forward_reference(x, w, I)
    check_h(h, g, u, G, U, H)
    for half, (v, mag) in enumerate(((g, G), (u, U))):
        err = H * E * mag
        if save == "bf16":
            got = f64(saved.data[:, half, :I])
            assert np.all(np.abs(got - v) <= err + F.bf16_ulp(v))
            continue
        codes, scale = O.checkpoint_int8(v)
        s = f64(saved.scale[:, half])
        for j in range(s.shape[1]):
            at = slice(128 * j, min(128 * (j + 1), I))
            worst = err[:, at].max(axis=1)
            assert np.all(np.abs(s[:, j] - scale[:, j]) <= worst / 127 + 2 * E * scale[:, j])
            c = f64(saved.data[:, half, at])
            step = s[:, j:j + 1]
            assert np.all(np.abs(c) <= 127)
            assert np.all(np.abs(c * step - v[:, at]) <= step * (0.5 + 256 * E) + err[:, at])
    dx, dw = ql.gated_ffn_backward(dh, x, w, saved)
    check_backward(dx, dw, dh, x, w, *kept(saved, I))


# tiles cut along K over pairs of CTAs: all of them (few tiles), the last ones after whole rounds, in
# the forward (with either checkpoint), dx (K = 2I) and dw (K = tokens)
@pytest.mark.parametrize("save", ["bf16", "int8"])
@pytest.mark.parametrize("M,H,I", [(300, 2048, 1024), (2000, 512, 520), (300, 512, 4096), (4096, 1600, 1400)])
def test_cut_tiles(ql, M, H, I, save):
    x, w, dh = make(M, H, I, seed=M + 2)
    h, saved = ql.gated_ffn(x, w, save=save)
    check_h(h, *forward_reference(x, w, I), H)
    dx, dw = ql.gated_ffn_backward(dh, x, w, saved)
    check_backward(dx, dw, dh, x, w, *kept(saved, I))
    for _ in range(3):  # the order of a sum does not depend on who finishes last
        h2, saved2 = ql.gated_ffn(x, w, save=save)
        dx2, dw2 = ql.gated_ffn_backward(dh, x, w, saved2)
        assert torch.equal(h2, h) and torch.equal(saved2.data[:, :, :I], saved.data[:, :, :I])
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("alpha,limit", [(1.0, 0.8), (1.7, 1.5), (-1.0, None), (1.0, 0.0)])
@pytest.mark.parametrize("M", [9, 65])
def test_activation_parameters(ql, M, alpha, limit):
    """The caps of both signs are hit; gradients vanish beyond them."""
    H, I = 128, 136
    x, w, dh = make(M, H, I, seed=5, gain=1.5)
    lim = np.inf if limit is None else limit
    g, u, G, U = forward_reference(x, w, I)
    check_h(ql.gated_ffn(x, w, swiglu_alpha=alpha, swiglu_limit=limit), g, u, G, U, H, alpha, lim)
    for save in ("bf16", "int8"):
        h, saved = ql.gated_ffn(x, w, swiglu_alpha=alpha, swiglu_limit=limit, save=save)
        check_h(h, g, u, G, U, H, alpha, lim)
        dx, dw = ql.gated_ffn_backward(dh, x, w, saved, swiglu_alpha=alpha, swiglu_limit=limit)
        check_backward(dx, dw, dh, x, w, *kept(saved, I), alpha, lim)


def test_strides_and_guard_columns(ql):
    M, H, I = 70, 136, 72
    x, w, dh = make(M, H, I, seed=7, pad=2)
    for m, save in ((4, None), (M, None), (M, "bf16")):  # the few-token kernel, twice; tcgen05
        wide = torch.full((m, I + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        ql.gated_ffn(x[:m], w, out=wide[:, 8:8 + I], save=save)
        check_h(wide[:, 8:8 + I], *forward_reference(x[:m], w, I), H)
        assert torch.all(wide[:, :8] == 7.0) and torch.all(wide[:, 8 + I:] == 7.0)
    _, saved = ql.gated_ffn(x, w, save="int8")
    wdx = torch.full((M, H + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    wdw = torch.full((2 * I + 2, H + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    ql.gated_ffn_backward(dh, x, w, saved, out_dx=wdx[:, 8:8 + H], out_dw=wdw[1:-1, 8:8 + H])
    check_backward(wdx[:, 8:8 + H], wdw[1:-1, 8:8 + H], dh, x, w, *kept(saved, I))
    assert torch.all(wdx[:, :8] == 7.0) and torch.all(wdx[:, 8 + H:] == 7.0)
    assert torch.all(wdw[:, :8] == 7.0) and torch.all(wdw[:, 8 + H:] == 7.0)
    assert torch.all(wdw[0] == 7.0) and torch.all(wdw[-1] == 7.0)


def test_one_gradient_alone_equals_both(ql):
    x, w, dh = make(140, 264, 136, seed=8)
    _, saved = ql.gated_ffn(x, w, save="bf16")
    dx, dw = ql.gated_ffn_backward(dh, x, w, saved)
    dx1, none = ql.gated_ffn_backward(dh, x, w, saved, need_dw=False)
    assert none is None and torch.equal(dx1, dx)
    none, dw1 = ql.gated_ffn_backward(dh, x, w, saved, need_dx=False)
    assert none is None and torch.equal(dw1, dw)
    dx2, dw2 = ql.gated_ffn_backward(dh, x, w, saved)  # the same bits every time
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_gradients_against_differences(ql):
    """Directional derivatives of sum(dh h) in 64 bits against the kernel's gradients: the 16-bit
    checkpoint moves g and u by 2^-8 relative, dg and du are rounded by 2^-8 and the outputs by 2^-8,
    so a random direction's derivative is within 4 * 2^-8 of the sum of magnitudes."""
    M, H, I = 40, 64, 48
    x, w, dh = make(M, H, I, seed=9)
    _, saved = ql.gated_ffn(x, w, save="bf16")
    dx, dw = ql.gated_ffn_backward(dh, x, w, saved)
    X, W, D = f64(x), f64(w), f64(dh)

    def loss(a, b):
        gu = a @ b.T
        return np.sum(D * O.gated(gu[:, :I], gu[:, I:]))

    r = np.random.default_rng(0)
    g, u = (X @ W.T)[:, :I], (X @ W.T)[:, I:]
    _, _, dgu = O.backward(D, X, W, g, u)
    for _ in range(4):
        vx, vw = r.normal(size=X.shape), r.normal(size=W.shape)
        e = 1e-5
        num = (loss(X + e * vx, W + e * vw) - loss(X - e * vx, W - e * vw)) / (2 * e)
        got = np.sum(f64(dx) * vx) + np.sum(f64(dw) * vw)
        mag = np.sum((np.abs(dgu) @ np.abs(W)) * np.abs(vx)) + np.sum((np.abs(dgu).T @ np.abs(X)) * np.abs(vw))
        assert abs(got - num) <= 4 * 2.0 ** -8 * mag


def test_zero_rows_and_tiny_values(ql):
    """A token of zeros keeps a checkpoint of zeros (scale 0); its gradients are finite."""
    x, w, dh = make(40, 64, 136, seed=10)
    x[3] = 0
    x[4] *= 2.0 ** -110
    h, saved = ql.gated_ffn(x, w, save="int8")
    assert torch.all(h[3] == 0) and torch.all(saved.data[3, :, :136] == 0) and torch.all(saved.scale[3] == 0)
    assert torch.all(saved.data[4, :, :136] == 0) and torch.all(saved.scale[4] == 0)
    dx, dw = ql.gated_ffn_backward(dh, x, w, saved)
    assert torch.all(dx[3] == 0) and torch.all(torch.isfinite(dw))


@pytest.mark.parametrize("save", ["bf16", "int8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_tokens_stay_in_their_rows(ql, save, bad):
    M, H, I = 48, 64, 136
    x, w, dh = make(M, H, I, seed=11)
    h0, s0 = ql.gated_ffn(x, w, save=save, swiglu_limit=3.0)
    dx0, _ = ql.gated_ffn_backward(dh, x, w, s0, swiglu_limit=3.0, need_dw=False)
    y = x.clone()
    y[7, 5] = bad
    h, s = ql.gated_ffn(y, w, save=save, swiglu_limit=3.0)
    dx, _ = ql.gated_ffn_backward(dh, y, w, s, swiglu_limit=3.0, need_dw=False)
    rest = [m for m in range(M) if m != 7]
    assert torch.equal(h[rest], h0[rest]) and torch.equal(dx[rest], dx0[rest])
    if bad != bad:
        assert torch.all(torch.isnan(h[7])) and torch.all(torch.isnan(dx[7]))
    elif save == "int8":  # an infinity in a group of 128 reads back as NaN
        assert torch.all(torch.isnan(dx[7]))


def test_offsets_past_32_bits(ql):
    """h and dh rows that start beyond 2^31 elements."""
    M, H, I, ld = 33000, 64, 64, 65544
    x, w, _ = make(M, H, I, seed=12)
    wide = torch.zeros(M, ld, dtype=torch.bfloat16, device="cuda")
    h, saved = ql.gated_ffn(x, w, save="int8", out=wide[:, :I])
    tail = slice(M - 300, M)
    check_h(h[tail], *forward_reference(x[tail], w, I), H)
    wide[:, :I] = torch.randn(M, I, device="cuda").to(torch.bfloat16)
    dx, _ = ql.gated_ffn_backward(wide[:, :I], x, w, saved, need_dw=False)
    part = type(saved)("int8", saved.data[tail], saved.scale[tail])
    check_backward(dx[tail], None, wide[tail, :I], x[tail], w, *kept(part, I))


def test_other_stream_and_graph(ql):
    x, w, dh = make(64, 128, 136, seed=13)
    h0, s0 = ql.gated_ffn(x, w, save="int8")
    dx0, dw0 = ql.gated_ffn_backward(dh, x, w, s0)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    h, s = ql.gated_ffn(x, w, save="int8", stream=st)
    dx, dw = ql.gated_ffn_backward(dh, x, w, s, stream=st)
    st.synchronize()
    assert torch.equal(h, h0) and torch.equal(dx, dx0) and torch.equal(dw, dw0)
    graph = torch.cuda.CUDAGraph()
    ws = ql.Workspace()
    ws.get(ql.workspace_bytes(ql.OP_GATED_FFN_BWD, 64, 136, 128))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        hg, sg = ql.gated_ffn(x, w, save="int8", workspace=ws)
        dxg, dwg = ql.gated_ffn_backward(dh, x, w, sg, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(hg, h0) and torch.equal(dxg, dx0) and torch.equal(dwg, dw0)


def test_streams_do_not_share_a_workspace(ql):
    """Backward passes on two streams, with the default workspaces, at the same time."""
    sets = [make(300, 512, 264, seed=20 + i) for i in range(2)]
    want = []
    for x, w, dh in sets:
        _, s = ql.gated_ffn(x, w, save="int8")
        want.append(ql.gated_ffn_backward(dh, x, w, s))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for explicit in (False, True):
        got = [None, None]
        for _ in range(10):
            for i, ((x, w, dh), st) in enumerate(zip(sets, streams)):
                if explicit:
                    _, s = ql.gated_ffn(x, w, save="int8", stream=st)
                    got[i] = ql.gated_ffn_backward(dh, x, w, s, stream=st)
                else:
                    with torch.cuda.stream(st):
                        _, s = ql.gated_ffn(x, w, save="int8")
                        got[i] = ql.gated_ffn_backward(dh, x, w, s)
        torch.cuda.synchronize()
        for (dx, dw), (rdx, rdw) in zip(got, want):
            assert torch.equal(dx, rdx) and torch.equal(dw, rdw)


def test_python_refusals(ql):
    x, w, dh = make(40, 64, 72)
    _, saved = ql.gated_ffn(x, w, save="int8")
    with pytest.raises(TypeError):
        ql.gated_ffn(x.float(), w)
    with pytest.raises(TypeError):
        ql.gated_ffn(x, w.float())
    with pytest.raises(TypeError):
        ql.gated_ffn(x, w.cpu())
    with pytest.raises(TypeError):
        ql.gated_ffn_backward(dh, x, w.cpu(), saved)
    with pytest.raises(ValueError):
        ql.gated_ffn_backward(dh, x, w, saved._replace(data=saved.data.cpu()))
    with pytest.raises(ValueError):
        ql.gated_ffn_backward(dh, x, w, saved._replace(scale=saved.scale.cpu()))
    with pytest.raises(TypeError):
        ql.gated_ffn(x, w, out=torch.empty(40, 80, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        ql.gated_ffn(x.t().contiguous().t(), w)  # a strided inner dimension
    with pytest.raises(ValueError):
        ql.gated_ffn(x, w[:-1])
    with pytest.raises(ValueError):
        ql.gated_ffn(x, w, save="fp8")
    with pytest.raises(TypeError):
        ql.gated_ffn_backward(dh[:, :64], x, w, saved)
    with pytest.raises(ValueError):
        ql.gated_ffn_backward(dh[:39], x[:39], w, saved)
    with pytest.raises(ql.QLError) as e:
        ql.gated_ffn_backward(dh, x, w, saved, need_dx=False, need_dw=False)
    assert e.value.status == 1


def test_timeout_is_reported_and_recoverable(ql):
    """With the wait limit at 0 the roles give up, the pair waits for its copies in flight, frees its
    tensor memory and returns; the status word says so and the next call is whole again."""
    x, w, dh = make(600, 512, 264, seed=14)
    ws = ql.Workspace()
    h0, s0 = ql.gated_ffn(x, w, save="bf16", workspace=ws)
    dx0, dw0 = ql.gated_ffn_backward(dh, x, w, s0, workspace=ws)
    torch.cuda.synchronize()
    assert ql.read_device_status(ws.buf) == (0, 0)
    ql.set_wait_limit(0)
    try:
        seen = False
        for _ in range(8):
            ql.gated_ffn(x, w, save="bf16", workspace=ws)
            ql.gated_ffn_backward(dh, x, w, s0, workspace=ws)
            st, flags = ql.read_device_status(ws.buf, clear=True)
            if flags & 1:
                seen = True
                break
    finally:
        ql.set_wait_limit(1 << 20)
    assert seen and st != 0
    ws.buf.zero_()  # tickets may be left mid-count: the workspace is initialised again
    h, s = ql.gated_ffn(x, w, save="bf16", workspace=ws)
    dx, dw = ql.gated_ffn_backward(dh, x, w, s, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(h, h0) and torch.equal(dx, dx0) and torch.equal(dw, dw0)
    assert ql.read_device_status(ws.buf) == (0, 0)
