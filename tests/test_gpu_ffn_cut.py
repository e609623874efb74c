"""The gated block's GEMMs where tiles are cut along the summed dimension over pairs of CTAs: all of a
GEMM's tiles or the last ones after whole rounds, in the forward with each checkpoint, in dx and in
dW13, with both gradients in one launch and in two that share the workspace.  The shapes are asserted
to be cut by the library's own plan.

Tolerances.  One by one as in test_gpu_ffn.py.  Of the whole output, ||got - exact|| / ||exact||:
  h         rounded once to bf16: errors spread evenly over +-2^-8 of a number's power of two, 0.8 to
            0.9 * 2^-9 of the norm over numbers of all leading digits; 2^-17 for the activation and
            2^-19 for fp32 sums: under 1.1 * 2^-9
  dx, dW13  that, and dg, du rounded to bf16 before the sums: as much again of terms whose errors are
            independent, a square root of two in all: under 2^-8
A step of 64 lost from one tile's sum is off by 0.0068 of the norm or more at the sizes here."""
import numpy as np
import pytest
import torch

from _util import gpu_lib
from oracle import ffn_oracle as O
from test_gpu_ffn import E, check_h, forward_reference, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def check_norm_h(h, x, w, I):
    gu = x.double() @ w.double().t()
    want = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
    assert off(h, want) < 1.1 * 2.0 ** -9
    return gu


def check_gradients(dx, dw, dh, x, w, saved, I):
    """From the checkpoint's values, all in 64 bits; the bound of every element as in test_gpu_ffn's
    check_backward."""
    v = saved.data[:, :, :I].float()
    if saved.mode == "int8":
        v = v * saved.scale.repeat_interleave(128, 2)[:, :, :I]
    g, u = v[:, 0].double(), v[:, 1].double()
    s, dh, x, w = torch.sigmoid(g), dh.double(), x.double(), w.double()
    dgu = torch.cat([dh * u * (s + g * s * (1 - s)), dh * g * s], 1)
    mag = torch.cat([(dh * u).abs() * (s + g.abs() * s), (dh * g).abs() * s], 1)
    err = 2.0 ** -8 * dgu.abs() + 2.0 ** -17 * mag
    for got, a, e, b in ((dx, dgu, err, w), (dw, dgu.t(), err.t(), x)):
        if got is None:
            continue
        want = a @ b
        assert off(got, want) < 2.0 ** -8
        tol = (e + a.shape[1] * E * (a.abs() + e)) @ b.abs() + 2.0 ** -8 * want.abs() + 2.0 ** -133
        assert bool(((got.double() - want).abs() <= tol).all())


# every form, all tiles cut and the last ones after a whole round
@pytest.mark.parametrize("M,H,I,save,whole", [(4962, 2304, 24, None, False), (4104, 4096, 520, None, True),
                                              (40, 4096, 72, "bf16", False), (4104, 4096, 520, "bf16", True),
                                              (40, 4096, 72, "int8", False), (4104, 4096, 520, "int8", True),
                                              (268, 3472, 5104, "int8", True)])
def test_forward(ql, M, H, I, save, whole):
    p = ql.gated_ffn_plan("forward", M, I, H, save=save)
    assert p.cut and (p.whole > 0) == whole
    x, w, _ = make(M, H, I, seed=M + 3)
    r = ql.gated_ffn(x, w, save=save)
    h, saved = (r, None) if save is None else r
    gu = check_norm_h(h, x, w, I)
    rows = torch.arange(0, M, max(1, M // 200), device="cuda")
    check_h(h[rows], *forward_reference(x[rows], w, I), H)
    if save == "bf16":
        assert off(torch.cat([saved.data[:, 0, :I], saved.data[:, 1, :I]], 1), gu) < 1.1 * 2.0 ** -9
    elif save == "int8":
        for half in range(2):
            v = gu[:, half * I:(half + 1) * I].cpu().numpy()
            codes, scale = O.checkpoint_int8(v)
            got_s = saved.scale[:, half].double().cpu().numpy()
            assert np.all(np.abs(got_s - scale) <= 2.0 ** -16 * scale)  # fp32 sums of 4096: 2^-19 of their norm
            step = np.repeat(got_s, 128, axis=1)[:, :I]
            got = saved.data[:, half, :I].double().cpu().numpy() * step
            assert np.all(np.abs(got - v) <= step * (0.5 + 2.0 ** -8))
    for _ in range(3):  # the sum does not depend on which part is the last
        r = ql.gated_ffn(x, w, save=save)
        h2, saved2 = (r, None) if save is None else r
        assert torch.equal(h2, h)
        if saved is not None:
            assert torch.equal(saved2.data[:, :, :I], saved.data[:, :, :I])


# (both gradients cut in one launch; dx after whole tiles, one launch; dW13 after whole tiles, one
# launch; two launches: all of dx, dx after whole tiles, both after whole tiles)
@pytest.mark.parametrize("save", ["bf16", "int8"])
@pytest.mark.parametrize("M,H,I,launches,dx_cut,dw_cut",
                         [(2406, 8, 1136, 1, True, True), (1, 6176, 1968, 1, True, False),
                          (2311, 8, 4800, 1, True, True), (5645, 8, 7440, 2, True, False),
                          (6899, 784, 2352, 2, True, False), (8439, 568, 6952, 2, True, True)])
def test_both_gradients(ql, M, H, I, launches, dx_cut, dw_cut, save):
    px, pw = (ql.gated_ffn_plan(g, M, I, H) for g in ("dx", "dw"))
    assert px.launches == pw.launches == launches
    assert (px.cut > 0, pw.cut > 0) == (dx_cut, dw_cut)
    x, w, dh = make(M, H, I, seed=M + 4)
    _, saved = ql.gated_ffn(x, w, save=save)
    dx, dw = ql.gated_ffn_backward(dh, x, w, saved)
    check_gradients(dx, dw, dh, x, w, saved, I)
    for _ in range(3):
        dx2, dw2 = ql.gated_ffn_backward(dh, x, w, saved)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


# one gradient alone is split over all pairs, with the other over a part of them: its sums may be cut
# elsewhere then, so the two ways agree within the tolerance, each with itself bit for bit
@pytest.mark.parametrize("M,H,I,gemm", [(40, 2056, 2448, "dx"), (3020, 296, 5288, "dw")])
def test_one_gradient_alone(ql, M, H, I, gemm):
    alone, both = (ql.gated_ffn_plan(gemm, M, I, H, both=b) for b in (False, True))
    assert alone.cut and (alone.cut, alone.parts) != (both.cut, both.parts)
    x, w, dh = make(M, H, I, seed=M + 5)
    _, saved = ql.gated_ffn(x, w, save="bf16")
    for kw in (dict(need_dw=gemm == "dw", need_dx=gemm == "dx"), {}):
        dx, dw = ql.gated_ffn_backward(dh, x, w, saved, **kw)
        check_gradients(dx, dw, dh, x, w, saved, I)
        dx2, dw2 = ql.gated_ffn_backward(dh, x, w, saved, **kw)
        assert dx is None or torch.equal(dx2, dx)
        assert dw is None or torch.equal(dw2, dw)
