"""Every zero point that a uint8 holds, exactly: whole-number activations and scales that are powers of
two make every sum a multiple of 2^-3 below 2^21, which fp32 holds, so that the outputs are the
rounded sums bit for bit, in whatever order they are added.  The gated block's g and u are then the
same numbers on 4-bit and on bf16 weights, and so is its output."""
import pytest
import torch

from _util import gpu_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


def weights(w, s, z, K, group):
    q = torch.stack((w[:, :K // 2] & 15, w[:, :K // 2] >> 4), 2).reshape(w.shape[0], K).double()
    at = torch.arange(K, device=w.device) // group
    return (q - z.double()[:, at]) * s.double()[:, at]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group", [32, 64, 128, 1024])
@pytest.mark.parametrize("M", [1, 5, 16, 32])
def test_zero_points_of_all_values(ql, M, group, dtype):
    N, K = 300, 1024
    g = torch.Generator(device="cuda").manual_seed(M + group)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, device="cuda", generator=g)

    x = ints(-3, 4, M, K).to(torch.bfloat16)
    w = ints(0, 256, N, K // 2).to(torch.uint8)
    s = (2.0 ** ints(-3, 1, N, K // group)).to(dtype)
    z = ((torch.arange(N * (K // group), device="cuda") * 7 + 128) % 256).reshape(N, -1).to(torch.uint8)
    assert z.unique().numel() == 256
    want = x.double() @ weights(w, s, z, K, group).t()
    assert float(want.abs().max()) < 2.0 ** 21
    assert torch.equal(ql.qlinear_int4(x, w, s, z, group=group), want.float().to(torch.bfloat16))
    s = (s.float() * 2.0 ** -12).to(dtype)  # (exact: fp16 keeps 2^-15 as a normal number)
    wide = torch.zeros(2, 152, K, dtype=torch.bfloat16, device="cuda")  # the weights themselves, exact in bf16
    wide[:, :N // 2] = weights(w, s, z, K, group).reshape(2, N // 2, K).to(torch.bfloat16)
    assert torch.equal(ql.gated_ffn_int4(x, w, s, z, group=group), ql.gated_ffn(x, wide.reshape(-1, K))[:, :N // 2])
