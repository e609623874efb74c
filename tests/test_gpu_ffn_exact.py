"""The gated block on bf16 weights with sums that fp32 holds exactly (whole-number activations and
weights times a power of two), so that a lost or doubled piece of K shows in every output: the few-token
kernel, the tcgen05 GEMM and the checkpoints have to agree bit for bit, and the bf16 checkpoint is the
rounded sum itself.

And the whole block's sizes (17408 x 5120), checked on sampled rows and columns.  Of those,
||got - exact|| / ||exact|| as in test_gpu_ffn_cut.py: h under 1.1 * 2^-9, dx and dW13 under 2^-8."""
import pytest
import torch

from _util import gpu_lib
from test_gpu_ffn import make
from test_gpu_ffn_cut import off

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


def exact_case(M, H, I):
    g = torch.Generator(device="cuda").manual_seed(M + H + I)
    x = torch.randint(-3, 4, (M, H), device="cuda", generator=g).to(torch.bfloat16)
    w = (torch.randint(-7, 8, (2 * I, H), device="cuda", generator=g) * 2.0 ** -9).to(torch.bfloat16)
    return x, w, x.double() @ w.double().t()


@pytest.mark.parametrize("M,H,I", [(1, 8200, 80), (7, 17408, 136), (16, 5120, 2440), (30, 2024, 2432), (40, 4096, 72),
                                   (300, 2056, 1000), (268, 3472, 5104), (4104, 4096, 520), (1000, 1032, 4104)])
def test_sums_are_whole(ql, M, H, I):
    x, w, gu = exact_case(M, H, I)
    h, saved = ql.gated_ffn(x, w, save="bf16")
    for half in range(2):
        assert torch.equal(saved.data[:, half, :I], gu[:, half * I:(half + 1) * I].float().to(torch.bfloat16))
    assert off(h, gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]) < 1.1 * 2.0 ** -9
    h8, saved8 = ql.gated_ffn(x, w, save="int8")
    assert torch.equal(h8, h)
    pad = torch.nn.functional.pad(gu.reshape(M, 2, I), (0, -I % 128)).reshape(M, 2, -1, 128)
    amax = pad.abs().amax(3)
    assert torch.equal(saved8.scale, amax.float() / torch.tensor(127.0, device="cuda"))  # rounded once in fp32
    code = saved8.data.reshape(M, 2, -1, 128).double()
    code[:, :, -1, (I - 1) % 128 + 1:] = 0  # past the last column: undefined
    # v (127 / amax) in fp32 is within 2^-23 of v / scale: off by one code only that near to a half
    assert bool(((code * amax[..., None] - 127 * pad).abs() <= (0.5 + 2.0 ** -15) * amax[..., None]).all())
    for rows in (slice(0, 1), slice(0, 13), slice(0, 32)):  # the few-token kernel; beyond 16 where I is small
        assert torch.equal(ql.gated_ffn(x[rows], w), h[rows])


def gradients(dh, g, u):
    s = torch.sigmoid(g)
    return torch.cat([dh * u * (s + g * s * (1 - s)), dh * g * s], 1)


def values(saved, rows, I):
    v = saved.data[rows, :, :I].float()
    if saved.mode == "int8":
        v = v * saved.scale[rows].repeat_interleave(128, 2)[:, :, :I]
    return v[:, 0].double(), v[:, 1].double()


@pytest.mark.parametrize("M", [1, 13, 1000])
def test_whole_block_forward_sampled(ql, M):
    I, H = 17408, 5120
    x, w, _ = make(M, H, I, seed=70)
    h = ql.gated_ffn(x, w)
    o = torch.cat([torch.tensor([0, 127, 128, I // 2, I - 129, I - 1]), torch.arange(5, I, 53)]).cuda()
    gu = x.double() @ torch.cat([w[o], w[I + o]]).double().t()
    g, u = gu[:, :len(o)], gu[:, len(o):]
    assert off(h[:, o], g * torch.sigmoid(g) * u) < 1.1 * 2.0 ** -9


@pytest.mark.parametrize("M,save", [(1000, "bf16"), (4096, "int8")])
def test_whole_block_step_sampled(ql, M, save):
    """Two GEMM launches; dx is cut after whole rounds."""
    I, H = 17408, 5120
    p = ql.gated_ffn_plan("dx", M, I, H)
    assert p.launches == 2 and p.cut and p.whole
    x, w, dh = make(M, H, I, seed=71)
    h, saved = ql.gated_ffn(x, w, save=save)
    dx, dw = ql.gated_ffn_backward(dh, x, w, saved)
    rows = torch.cat([torch.tensor([0, 255, 256, M - 1]), torch.arange(3, M, M // 28)]).cuda()
    gu = x[rows].double() @ w.double().t()
    assert off(h[rows], gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]) < 1.1 * 2.0 ** -9
    g, u = values(saved, rows, I)
    if save == "int8":  # half a step of 127, and what fp32 sums of 5120 products lose: under 2^-12 of a step
        step = saved.scale[rows].double().repeat_interleave(128, 2)[:, :, :I]
        assert bool(((g - gu[:, :I]).abs() <= (0.5 + 2.0 ** -8) * step[:, 0]).all())
        assert bool(((u - gu[:, I:]).abs() <= (0.5 + 2.0 ** -8) * step[:, 1]).all())
    got = dx[rows]
    want = gradients(dh[rows].double(), g, u) @ w.double()
    assert off(got, want) < 2.0 ** -8
    for at in (slice(0, 256), slice(2560, 2816), slice(H - 256, H)):  # and by columns of a tile
        assert off(got[:, at], want[:, at]) < 2.0 ** -8
    o = torch.cat([torch.tensor([0, 255, 256, I - 1]), torch.arange(7, I, 311)]).cuda()
    g, u = values(saved, slice(None), I)
    dgu = gradients(dh[:, o].double(), g[:, o], u[:, o])
    assert off(dw[torch.cat([o, I + o])], dgu.t() @ x.double()) < 2.0 ** -8
