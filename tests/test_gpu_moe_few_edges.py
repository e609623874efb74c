"""Edges of the mixture-of-experts layers for a few tokens: what the debug output holds for padding,
4-bit layers on tokens of any magnitude, what is rounded in the 8-bit layer's down, up to 1024 experts, experts
of many tokens.  Tolerances are those of test_gpu_moe_few where no others are derived.  One workspace for
these calls and the library's other ones: test_gpu_workspace_sharing_more.py."""
import numpy as np
import pytest
import torch

from _util import bits_of, gpu_lib
from oracle import formats as F
from oracle import moe_few_oracle as MO
from test_gpu_moe_few import Layer, check, rebuild, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


@pytest.mark.parametrize("M", [1, 5, 40])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
def test_debug_h_of_padding_is_zero(ql, fmt, M):
    """A pair without an expert has zeros in the debug h, whatever an earlier call left in the workspace."""
    E, topk, H, I = 7, 3, 224, 96
    layer = Layer(fmt, E, H, I, seed=M)
    x, ws = tokens(M, H, seed=M, fmt=fmt), ql.Workspace("cuda")
    g = np.random.default_rng(M)
    ids = np.stack([g.permutation(E)[:topk] for _ in range(M)]).astype(np.int32)
    w = g.random((M, topk)).astype(np.float32)
    how = dict(topk_weights=torch.from_numpy(w).cuda(), workspace=ws, debug=True)
    full = layer(ql, x, topk_ids=torch.from_numpy(ids).cuda(), **how)
    check(layer, x, full, ids=ids, weights=w.astype(np.float64))
    assert full[3].any(dim=1).all()
    some = ids.copy()
    some[:, 1] = (-1, E, 1 << 30)[M % 3]
    some[M // 2] = -1
    got = layer(ql, x, topk_ids=torch.from_numpy(some).cuda(), **how)
    check(layer, x, got, ids=some, weights=w.astype(np.float64))
    off = torch.from_numpy(((some < 0) | (some >= E)).reshape(-1)).cuda()
    assert not got[3][off].any()
    assert torch.equal(got[3][~off], full[3][~off])
    ws.buf[256 + (1 << 20):] = 0xFF  # every 16-bit number a NaN
    none = layer(ql, x, topk_ids=torch.full((M, topk), -1, dtype=torch.int32).cuda(), **how)
    assert not none[3].any() and not none[0].any()


@pytest.mark.parametrize("M,H", [(1, 256), (6, 288), (24, 4096)])
@pytest.mark.parametrize("group,zeros,limit", [(32, True, 1.5), (64, False, None), (128, True, None), (128, False, 1.5)])
@pytest.mark.parametrize("power", [100, 62, -78])
def test_int4_tokens_of_any_magnitude(ql, M, H, group, zeros, limit, power):
    """x far from one and weights as far on the other side: sums of ordinary size.  Beside large tokens half
    stay ordinary, and their sums, 2^-power of the others', count like any."""
    layer = Layer("int4", 4, H, 64, seed=M + group, group=group, zeros=True)
    s13 = layer.args[1]
    if not zeros:
        for z in layer.zero_args:
            z.fill_(8)
    layer.args[1] = (s13.double() * 2.0 ** -power).to(torch.bfloat16)
    rebuild(layer)
    if not zeros:
        layer.zero_args = [None, None]
    x = (tokens(M, H, seed=M).double() * 2.0 ** power).to(torch.bfloat16)
    if power > 0:  # (with weights of 2^78 ordinary tokens' h is infinite by the definition)
        x[1::2] = tokens(M, H, seed=M + 1)[1::2]
    logits = torch.randn(M, 4, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    got = layer(ql, x, router_logits=logits, topk=2, swiglu_limit=limit, debug=True)
    assert got[3].view(M, 2, 64)[::2].any(dim=2).all()
    check(layer, x, got, logits=logits, topk=2, limit=limit or np.inf)


@pytest.mark.parametrize("M,H", [(1, 256), (6, 288), (24, 4096)])
@pytest.mark.parametrize("group", [32, 128])
def test_int4_codes_at_their_zero_point_are_nothing(ql, M, H, group):
    """Rows whose codes all equal their zero points give zero exactly, however large x."""
    layer = Layer("int4", 3, H, 64, seed=M, group=group)
    layer.args[0][:, 64:] = 0x55  # the up rows
    layer.zero_args[0][:, 64:] = 5
    rebuild(layer)
    x = tokens(M, H, seed=M) * 100
    logits = torch.randn(M, 3, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    y, _, _, h, _ = layer(ql, x, router_logits=logits, topk=2, debug=True)
    assert not h.any() and not y.any()


@pytest.mark.parametrize("M,H", [(1, 32768), (2, 32768), (3, 32736), (19, 4096), (20, 4096)])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (256, False)])
def test_int4_tokens_that_just_fit_in_shared_memory(ql, M, H, group, zeros):
    layer = Layer("int4", 2, H, 32, seed=M, group=group, zeros=zeros, pad=1)
    x = tokens(M, H, seed=M, pad=1)
    logits = torch.randn(M, 2, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    check(layer, x, layer(ql, x, router_logits=logits, topk=2, debug=True), logits=logits, topk=2)


def int8_down(layer, h, ids, weights):
    """(y, how far fp32 may be off) of moe_int8's down on the kernel's own h.

    An expert's whole-number sums over units of 128 k are exact, and so are those of the runs of units that a
    warp adds (at most 1024 k).  A run's sum meets the channel's scale (one rounding) and the weight times the
    scale of h (one rounding to make it, one by the multiply-add that adds it).  A token has U = topk *
    ceil(I / 128) units, so no more than U runs, U parts of warps and U parts of CTAs that are not zero: 3 U
    additions and 2 roundings of a term, each by 2^-24 of the units' magnitudes."""
    q, s = MO.codes(h)
    M, topk = ids.shape
    w2, s2 = layer.values[1], layer.scales[1]
    y, a = np.zeros((M, layer.H)), np.zeros((M, layer.H))
    for p, e in enumerate(ids.reshape(-1)):
        if 0 <= e < layer.E:
            f = weights.reshape(-1)[p] * s[p] * s2[e]
            for k in range(0, layer.I, 128):
                unit = w2[e][:, k:k + 128] @ q[p, k:k + 128]
                y[p // topk] += f * unit
                a[p // topk] += np.abs(f * unit)
    return y, (3 * topk * -(-layer.I // 128) + 2) * 2.0 ** -24 * a


@pytest.mark.parametrize("M,E,topk,H,I", [(1, 8, 2, 256, 128), (1, 6, 6, 1024, 2080), (7, 5, 3, 544, 1056),
                                          (24, 4, 2, 288, 4096), (64, 3, 3, 96, 608)])
def test_int8_down_rounds_runs_not_products(ql, M, E, topk, H, I):
    layer = Layer("int8", E, H, I, seed=I)
    x = tokens(M, H, seed=I, fmt="int8")
    g = np.random.default_rng(I)
    ids = np.stack([g.permutation(E)[:topk] for _ in range(M)]).astype(np.int32)
    w = g.standard_normal((M, topk)).astype(np.float32)
    y, _, _, h, _ = layer(ql, x, topk_ids=torch.from_numpy(ids).cuda(), topk_weights=torch.from_numpy(w).cuda(), debug=True)
    ref, off = int8_down(layer, F.bf16_to_f64(bits_of(h)), ids, w.astype(np.float64))
    assert (np.abs(F.bf16_to_f64(bits_of(y)) - ref) <= off + F.bf16_ulp(np.abs(ref) + off) / 2).all()


@pytest.mark.parametrize("M,H,I", [(1, 512, 2080), (9, 256, 1056), (40, 160, 608)])
def test_int8_down_of_opposite_weights(ql, M, H, I):
    """Two experts of equal weights, w and -w: what is left are the roundings of runs, and no bf16 rounding
    of a larger result hides them."""
    layer = Layer("int8", 4, H, I, seed=I)
    for a in (*layer.args, *layer.values, *layer.scales):
        a[2:] = a[:2]
    x = tokens(M, H, seed=I, fmt="int8")
    ids = np.tile(np.array([[0, 2, 3, 1]], np.int32), (M, 1))
    w = np.random.default_rng(1).random((M, 2)).astype(np.float32)
    w = np.stack((w[:, 0], -w[:, 0], w[:, 1], -w[:, 1]), axis=1)
    y, _, _, h, _ = layer(ql, x, topk_ids=torch.from_numpy(ids).cuda(), topk_weights=torch.from_numpy(w).cuda(), debug=True)
    hv = h.view(M, 4, I)
    assert torch.equal(hv[:, 0], hv[:, 1]) and torch.equal(hv[:, 2], hv[:, 3])
    ref, off = int8_down(layer, F.bf16_to_f64(bits_of(h)), ids, w.astype(np.float64))
    assert (np.abs(ref) <= 2.0 ** -40 * off / 2.0 ** -24).all()
    assert (np.abs(F.bf16_to_f64(bits_of(y))) <= off * (1 + 2.0 ** -8)).all()


@pytest.mark.parametrize("E", [257, 512, 513, 1024])
@pytest.mark.parametrize("M,topk", [(1, 8), (1, 16), (5, 3), (33, 16)])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
def test_many_experts(ql, fmt, E, M, topk):
    """Every form of the router, with tied logits; a wrong pairing of ids and weights would show in y."""
    layer = Layer(fmt, E, 64, 32, seed=E)
    x = tokens(M, 64, seed=E, fmt=fmt)
    g = torch.Generator().manual_seed(E + M)
    logits = (torch.randint(-9, 10, (M, E), generator=g) / 4).to(torch.bfloat16).cuda()
    logits[0, E - 1] = 3.0
    check(layer, x, layer(ql, x, router_logits=logits, topk=topk, renormalize=E % 2 == 1, debug=True), logits=logits,
          topk=topk, renorm=E % 2 == 1)


@pytest.mark.parametrize("M", [1, 4, 20])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
def test_given_ids_of_the_last_experts_that_repeat(ql, fmt, M):
    E = 1024
    layer = Layer(fmt, E, 64, 32, seed=3)
    x = tokens(M, 64, seed=4, fmt=fmt)
    g = np.random.default_rng(M)
    ids = g.choice([E - 1, E - 2, E - 17, 0, -1, E], (M, 16), p=[0.4, 0.2, 0.1, 0.1, 0.1, 0.1]).astype(np.int32)
    ids[0] = E - 1
    w = g.standard_normal((M, 16)).astype(np.float32)
    got = layer(ql, x, topk_ids=torch.from_numpy(ids).cuda(), topk_weights=torch.from_numpy(w).cuda(), debug=True)
    check(layer, x, got, ids=ids, weights=w.astype(np.float64))


@pytest.mark.parametrize("M,H,I", [(40, 2080, 96), (64, 1056, 1056), (24, 4096, 160), (17, 96, 2080)])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
def test_experts_of_many_tokens_on_cut_sums(ql, fmt, M, H, I):
    """Two of three experts and ids that repeat: an expert has up to 64 tokens two times each, and both launches cut
    its K over several warps and CTAs."""
    layer = Layer(fmt, 3, H, I, seed=M, group=64)
    x = tokens(M, H, seed=M, fmt=fmt)
    g = np.random.default_rng(M)
    ids = g.integers(0, 2, (M, 3)).astype(np.int32)
    ids[::5, 1] = -1
    w = g.standard_normal((M, 3)).astype(np.float32)
    got = layer(ql, x, topk_ids=torch.from_numpy(ids).cuda(), topk_weights=torch.from_numpy(w).cuda(), debug=True)
    check(layer, x, got, ids=ids, weights=w.astype(np.float64))
