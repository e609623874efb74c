"""Mixture-of-experts layers for a few tokens on bf16, 8-bit and 4-bit weights, against the 64-bit
definition.

Tolerances.  A product of two bf16 values, of a bf16 value and q - z, and of two codes is exact in fp32.
Each of the K additions of an fp32 sum rounds or truncates by at most 2^-23 of the sum of magnitudes;
sums of codes are exact, and their conversion and two scales put 3 roundings of 2^-24 on them.  h is
compared with the definition on x, y with the definition on the kernel's own h, ids and weights; h and y
are rounded to bf16 (half an ulp; 1 is allowed).  Codes are exact: ties fall as fp32 divisions let them."""
import numpy as np
import pytest
import torch

from _util import bits_of, gpu_lib
from oracle import ffn_oracle as O
from oracle import formats as F
from oracle import moe_few_oracle as MO
from oracle import qlinear_oracle as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


class Layer:
    """Weights of one layer: the arguments of a call and their 64-bit values."""

    def __init__(self, fmt, E, H, I, seed=0, group=128, zeros=True, dtype=torch.bfloat16, pad=0):
        self.fmt, self.E, self.H, self.I, self.group = fmt, E, H, I, group
        g = torch.Generator().manual_seed(seed)
        self.args, self.zero_args, self.values, self.scales = [], [], [], []
        for rows, k in ((2 * I, H), (H, I)):
            if fmt == "bf16":
                w = torch.full((E, rows, k + 8 * pad), float("nan"))
                w[..., :k] = torch.randn(E, rows, k, generator=g) / k ** 0.5
                w = w.to(torch.bfloat16)
                self.args.append(w.cuda())
                self.values.append(w[..., :k].double().numpy())
            elif fmt == "int8":
                w = torch.randint(-128, 128, (E, rows, k + 16 * pad), generator=g, dtype=torch.int8)
                s = (torch.rand(E, rows, generator=g) + 0.5) / (73 * k ** 0.5)
                self.args += [w.cuda(), s.cuda()]
                self.values.append(w[..., :k].double().numpy())  # whole numbers: exact sums; scales apart
                self.scales.append(s.double().numpy())
            else:
                groups = -(-k // group)
                w = torch.randint(0, 256, (E, rows, k // 2 + 16 * pad), generator=g, dtype=torch.uint8)
                s = ((torch.rand(E, rows, groups + pad, generator=g) + 0.1) * 0.4 / k ** 0.5).to(dtype)
                s[..., groups:] = float("nan")  # never read
                z = torch.randint(0, 16, (E, rows, groups + pad), generator=g, dtype=torch.uint8) if zeros else None
                self.args += [w.cuda(), s.cuda()]
                self.zero_args.append(None if z is None else z.cuda())
                self.values.append(np.stack([O.int4_dequant(w[e].numpy(), s[e].double().numpy(),
                                                            None if z is None else z[e].numpy(), k, group)
                                             for e in range(E)]))

    def __call__(self, ql, x, **kw):
        args = [a[..., :self.H] if i == 0 and self.fmt != "int4" else a for i, a in enumerate(self.args)]
        if self.fmt != "int4":  # the padding is not part of the tensors
            j = 1 if self.fmt == "bf16" else 2
            args[j] = args[j][..., :self.I]
        else:
            kw["group"] = self.group
        return getattr(ql, "moe_" + self.fmt)(x, *args, *self.zero_args, **kw)


def tokens(M, H, seed=0, pad=0, fmt="bf16"):
    g = torch.Generator().manual_seed(seed + 1000)
    x = torch.full((M, H + 8 * pad), float("nan"), dtype=torch.bfloat16)
    v = torch.randn(M, H, generator=g) * torch.where(torch.rand(H, generator=g) < 0.02, 6.0, 1.0)
    v[:, 1::7] = v.abs().amax(dim=1, keepdim=True) / 2  # ties: 63.5 steps
    x[:, :H] = v.to(torch.bfloat16)
    return x.cuda()[:, :H]


def check(layer, x, got, ids=None, weights=None, logits=None, topk=None, renorm=False, alpha=1.0, limit=np.inf):
    y, gids, gw, h, path = got
    assert path == "moe_" + layer.fmt
    M = x.shape[0]
    if logits is not None:
        ids, weights = Q.route_topk(bits_of(logits), topk, renorm)
        assert np.array_equal(gids.cpu().numpy(), ids)
        assert np.allclose(gw.cpu().numpy(), weights, rtol=2e-6, atol=0)
        weights = gw.cpu().numpy().astype(np.float64)
    used = ((ids >= 0) & (ids < layer.E)).reshape(-1)
    xv = x.double().cpu().numpy()
    w13, w2 = layer.values
    if layer.fmt == "int8":
        q, s = MO.codes(xv)
        gu = np.concatenate(MO.gate_up(q, w13, ids)[:2], axis=1)
        at = np.where(used, ids.reshape(-1), 0)
        gu *= np.repeat(s, ids.shape[1], axis=0) * layer.scales[0][at]
        g, u = np.split(gu, 2, axis=1)
        G, U = np.abs(g), np.abs(u)
        w2 = w2 * layer.scales[1][:, :, None]
    else:
        g, u, G, U = MO.gate_up(xv, w13, ids)
    eps = 2.0 ** -22 if layer.fmt == "int8" else layer.H * 2.0 ** -23
    ref, off = MO.activation(g, u, eps * G, eps * U, alpha, limit)
    hv = F.bf16_to_f64(bits_of(h))
    bad = ~(np.abs(hv - ref) <= off + F.bf16_ulp(ref))[used]
    assert not bad.any(), ("h", int(bad.sum()), bad.size, np.argwhere(bad)[:4].tolist())
    hv = np.where(used[:, None], hv, 0.0)
    if layer.fmt == "int8":
        q, s = MO.codes(hv)
        hv = q * s
    ref, a = MO.down(hv, w2, ids, weights)
    # fp32 sums over the experts' k, the weighted sum over experts, and (8-bit) three roundings a term
    tol = (layer.I + 2 * ids.shape[1] + 8) * 2.0 ** -23 * a + F.bf16_ulp(ref)
    yv = F.bf16_to_f64(bits_of(y))
    bad = ~(np.abs(yv - ref) <= tol)
    assert not bad.any(), ("y", int(bad.sum()), bad.size, np.argwhere(bad)[:4].tolist())


CASES = [  # M, E, topk, H, I
    (1, 8, 2, 256, 128), (1, 1, 1, 32, 32), (2, 5, 3, 96, 64), (3, 256, 8, 512, 160), (5, 3, 3, 160, 224),
    (8, 16, 4, 1056, 96), (9, 4, 2, 288, 352), (13, 60, 4, 544, 96), (16, 4, 4, 128, 1056), (33, 7, 1, 64, 96),
    (64, 12, 5, 96, 32), (64, 40, 16, 32, 64)]


@pytest.mark.parametrize("M,E,topk,H,I", CASES)
@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
def test_moe_matches_the_definition(ql, fmt, M, E, topk, H, I):
    i = M + E
    layer = Layer(fmt, E, H, I, seed=i, group=(32, 64, 128, 256)[i % 4], zeros=i % 2 == 0,
                  dtype=(torch.bfloat16, torch.float16)[i % 3 % 2], pad=i % 3)
    x = tokens(M, H, seed=i, pad=i % 3, fmt=fmt)
    logits = torch.randn(M, E, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda()
    renorm, limit = i % 2 == 1, (None, 1.5)[i % 2]
    got = layer(ql, x, router_logits=logits, topk=topk, renormalize=renorm, swiglu_limit=limit, debug=True)
    check(layer, x, got, logits=logits, topk=topk, renorm=renorm, limit=limit or np.inf)


@pytest.mark.parametrize("fmt,H,I", [("bf16", 1032, 520), ("bf16", 8, 8), ("int8", 1040, 528), ("int8", 16, 16)])
def test_odd_sizes(ql, fmt, H, I):
    layer = Layer(fmt, 6, H, I, seed=H)
    x = tokens(4, H, seed=H, fmt=fmt)
    logits = torch.randn(4, 6, generator=torch.Generator().manual_seed(H)).to(torch.bfloat16).cuda()
    check(layer, x, layer(ql, x, router_logits=logits, topk=3, debug=True, swiglu_alpha=1.3), logits=logits, topk=3,
          alpha=1.3)


@pytest.mark.parametrize("group,zeros,dtype", [(32, True, torch.float16), (32, False, torch.bfloat16),
                                               (64, True, torch.bfloat16), (128, False, torch.float16),
                                               (128, True, torch.bfloat16), (1 << 20, True, torch.bfloat16)])
def test_int4_groups(ql, group, zeros, dtype):
    layer = Layer("int4", 5, 480, 416, seed=group % 97, group=group, zeros=zeros, dtype=dtype, pad=1)
    if zeros:  # zero points are 0..255
        for z in layer.zero_args:
            z[0, 0, 0] = 200
        rebuild(layer)
    x = tokens(6, 480, seed=3)
    logits = torch.randn(6, 5, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    check(layer, x, layer(ql, x, router_logits=logits, topk=2, debug=True), logits=logits, topk=2)


def rebuild(layer):
    """The 64-bit values of a 4-bit layer's tensors as they are now."""
    for n, k in ((0, layer.H), (1, layer.I)):
        w, s, z = layer.args[2 * n].cpu().numpy(), layer.args[2 * n + 1].double().cpu().numpy(), layer.zero_args[n].cpu().numpy()
        layer.values[n] = np.stack([O.int4_dequant(w[e], s[e], z[e], k, layer.group) for e in range(layer.E)])


@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
def test_given_ids_padding_and_repeats(ql, fmt):
    layer = Layer(fmt, 9, 192, 96, seed=4)
    x = tokens(5, 192, seed=5, fmt=fmt)
    ids = np.array([[0, 8, 3], [-1, 4, 9], [-1, -1, -1], [2, 2, 2], [5, 1 << 30, 5]], np.int32)
    w = np.array([[0.5, 0.25, 1.0], [9.0, 0.5, 9.0], [1.0, 1.0, 1.0], [0.125, 0.5, -0.25], [0.0, 3.0, 0.75]], np.float32)
    got = layer(ql, x, topk_ids=torch.from_numpy(ids).cuda(), topk_weights=torch.from_numpy(w).cuda(), debug=True)
    check(layer, x, got, ids=ids, weights=w.astype(np.float64))
    assert np.array_equal(got[1].cpu().numpy(), np.where((ids < 0) | (ids >= 9), -1, ids))
    assert not got[0][2].any()
    none = layer(ql, x, topk_ids=torch.full((5, 3), -1, dtype=torch.int32).cuda(), topk_weights=torch.ones(5, 3).cuda(),
                 out=torch.full((5, 192), 7.0, dtype=torch.bfloat16, device="cuda"))
    assert not none.any()


def test_ties_and_extreme_logits(ql):
    layer = Layer("bf16", 40, 64, 32, seed=8)
    x = tokens(4, 64)
    logits = torch.zeros(4, 40)
    logits[0, 10:] = -float("inf")  # masked experts
    logits[1, 7:9] = torch.finfo(torch.bfloat16).max
    logits[2] = torch.finfo(torch.bfloat16).min
    logits[3, ::2] = -0.0
    logits = logits.to(torch.bfloat16).cuda()
    check(layer, x, layer(ql, x, router_logits=logits, topk=6, debug=True), logits=logits, topk=6)


@pytest.mark.parametrize("M", [1, 9, 20])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
def test_a_token_with_nan_leaves_the_others(ql, fmt, M):
    layer = Layer(fmt, 6, 160, 96, seed=2)
    x = tokens(M, 160, seed=6, fmt=fmt)
    at = M // 2
    logits = torch.randn(M, 6, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    clean = layer(ql, x, router_logits=logits, topk=3)
    for bad in (float("nan"), float("inf")):
        dirty = x.clone()
        dirty[at, 77] = bad
        y = layer(ql, dirty, router_logits=logits, topk=3)
        assert torch.equal(torch.cat((y[:at], y[at + 1:])), torch.cat((clean[:at], clean[at + 1:])))
        assert y[at].isnan().all()
    zero = x.clone()
    zero[at] = 0
    assert not layer(ql, zero, router_logits=logits, topk=3)[at].any()


@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
def test_workspace_is_left_zero_and_results_repeat(ql, fmt):
    layer = Layer(fmt, 32, 1024, 320, seed=11)
    ws = ql.Workspace("cuda")
    logits = torch.randn(40, 32, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    x = tokens(40, 1024, seed=7, fmt=fmt)
    first = {}
    for M in (12, 1, 7, 40, 12, 1, 7, 40):
        y = layer(ql, x[:M], router_logits=logits[:M], topk=4, workspace=ws)
        assert not ws.buf[:256 + (1 << 20)].any()
        assert torch.equal(first.setdefault(M, y), y)


def test_full_size_layers(ql):
    topk, H, I = 8, 4096, 2048
    for fmt, M in (("int4", 1), ("int8", 2), ("bf16", 1)):
        layer = Layer(fmt, 12, H, I, seed=1, zeros=False)
        ids = np.stack([np.random.default_rng(m).permutation(12)[:topk] for m in range(M)]).astype(np.int32)
        w = np.random.default_rng(5).random((M, topk)).astype(np.float32)
        x = tokens(M, H, seed=9, fmt=fmt)
        got = layer(ql, x, topk_ids=torch.from_numpy(ids).cuda(), topk_weights=torch.from_numpy(w).cuda(), debug=True)
        check(layer, x, got, ids=ids, weights=w.astype(np.float64))


@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("M,E,topk,H,I", [(16, 3, 2, 4096, 64), (8, 3, 2, 8224, 32), (12, 2, 2, 96, 8224)])
def test_rows_too_long_for_shared_memory(ql, fmt, M, E, topk, H, I):
    layer = Layer(fmt, E, H, I, seed=M, group=64)
    x = tokens(M, H, seed=M, fmt=fmt)
    logits = torch.randn(M, E, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    check(layer, x, layer(ql, x, router_logits=logits, topk=topk, debug=True), logits=logits, topk=topk)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("M,E,topk,H,I", [(4, 2, 1, 32768, 32), (4, 2, 2, 32768, 32), (3, 3, 2, 32736, 416), (21, 3, 3, 24608, 160)])
def test_wide_outputs(ql, fmt, M, E, topk, H, I):
    """Down: warps that hold whole tiles, parts of two, and both."""
    layer = Layer(fmt, E, H, I, seed=M, group=128)
    x = tokens(M, H, seed=M, fmt=fmt)
    logits = torch.randn(M, E, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    check(layer, x, layer(ql, x, router_logits=logits, topk=topk, debug=True), logits=logits, topk=topk)


@pytest.mark.parametrize("M,H", [(12, 4096), (18, 4096), (24, 2080), (20, 2080)])
@pytest.mark.parametrize("group,zeros", [(32, True), (32, False), (128, True), (128, False)])
def test_int4_many_tokens_in_shared_memory(ql, M, H, group, zeros):
    layer = Layer("int4", 4, H, 96, seed=M, group=group, zeros=zeros)
    x = tokens(M, H, seed=M)
    logits = torch.randn(M, 4, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    check(layer, x, layer(ql, x, router_logits=logits, topk=2, debug=True), logits=logits, topk=2)


@pytest.mark.parametrize("M", [1, 6, 24])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
def test_graphs_streams_and_threads(ql, fmt, M):
    """Captured graphs replayed in any order and against eager calls, a call on a given stream, and host
    threads on one stream give what one call gives."""
    import threading
    layers = [Layer(fmt, 16, 288, 160, seed=s) for s in (1, 2)]
    x = tokens(M, 288, seed=8, fmt=fmt)
    logits = torch.randn(M, 16, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    run = [lambda l=l, **kw: l(ql, x, router_logits=logits, topk=4, **kw) for l in layers]
    want = [r() for r in run]
    graphs = []
    for r in run:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            first = r()
            out = (first, r(debug=True))
        graphs.append((g, out))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for order in ((0, 1), (1, 0), (1, 1, 0)):
        for i in order:
            graphs[i][0].replay()
            there = run[1 - i](stream=side)
            torch.cuda.synchronize()
            assert torch.equal(graphs[i][1][0], want[i]) and torch.equal(graphs[i][1][1][0], want[i])
            assert torch.equal(there, want[1 - i])
    with torch.cuda.stream(side):  # two graphs at once, each with memory of its own
        graphs[0][0].replay()
    graphs[1][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g[1][0], w) for g, w in zip(graphs, want))
    bad = []

    def thread(i):
        for _ in range(20):
            if not torch.equal(run[i % 2](), want[i % 2]):
                bad.append(i)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_outputs_and_refusals(ql):
    layer = Layer("int8", 4, 64, 32, seed=5)
    x = tokens(3, 64, fmt="int8")
    logits = torch.randn(3, 4, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    want = layer(ql, x, router_logits=logits, topk=2)
    wide = torch.full((5, 96), 3.0, dtype=torch.bfloat16, device="cuda")
    layer(ql, x, router_logits=logits, topk=2, out=wide[1:4, 16:80])
    assert torch.equal(wide[1:4, 16:80], want)
    wide[1:4, 16:80] = 3.0
    assert (wide == 3.0).all()
    w13, s13, w2, s2 = layer.args
    ids, wt = torch.zeros(3, 2, dtype=torch.int32).cuda(), torch.ones(3, 2).cuda()
    for args, kw in [((x.cpu(), w13, s13, w2, s2), dict(router_logits=logits, topk=2)),
                     ((x, w13.cpu(), s13, w2, s2), dict(router_logits=logits, topk=2)),
                     ((x, w13, s13.cpu(), w2, s2), dict(router_logits=logits, topk=2)),
                     ((x, w13, s13, w2, s2), dict(router_logits=logits.cpu(), topk=2)),
                     ((x, w13, s13, w2, s2), dict(router_logits=logits.float(), topk=2)),
                     ((x, w13, s13, w2, s2), dict(topk=2)),
                     ((x, w13, s13, w2, s2), dict(router_logits=logits, topk_ids=ids, topk_weights=wt)),
                     ((x, w13, s13, w2, s2), dict(topk_ids=ids)),
                     ((x, w13, s13, w2, s2), dict(topk_ids=ids.long(), topk_weights=wt)),
                     ((x, w13, s13, w2, s2), dict(topk_ids=ids[:2], topk_weights=wt)),
                     ((x, w13[:, :63], s13, w2, s2), dict(router_logits=logits, topk=2)),
                     ((x, w13, s13[:, :60], w2, s2), dict(router_logits=logits, topk=2)),
                     ((x, w13, s13, w2[:3], s2), dict(router_logits=logits, topk=2)),
                     ((x, w13, s13, w2, s2), dict(router_logits=logits, topk=5)),
                     ((x, w13, s13, w2, s2), dict(router_logits=logits, topk=0)),
                     ((x, w13, s13, w2, s2), dict(router_logits=logits, topk=2, swiglu_limit=-1.0)),
                     ((x.t(), w13, s13, w2, s2), dict(router_logits=logits, topk=2)),
                     ((x[:0], w13, s13, w2, s2), dict(router_logits=logits[:0], topk=2)),
                     ((x.repeat(22, 1), w13, s13, w2, s2), dict(router_logits=logits.repeat(22, 1), topk=2)),
                     ((x, w13, s13, w2, s2), dict(router_logits=logits, topk=2, out=wide[:3, :63]))]:
        with pytest.raises((TypeError, ValueError, ql.QLError)):
            ql.moe_int8(*args, **kw)
