"""quantize_int8 and qlinear_int8 beside qlinear_int8_w8a8: the same codes, scales and results bit for bit for
finite tokens down to the smallest, and what a NaN or an infinity in a token gives."""
import pytest
import torch

from _util import gpu_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


def weights(N, K):
    g = torch.Generator().manual_seed(N)
    return (torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda(), (torch.rand(N, generator=g) + 0.5).cuda())


@pytest.mark.parametrize("M", [1, 4, 16, 30, 260])
@pytest.mark.parametrize("power", [0, 100, 112, 118, 126])
def test_small_tokens(ql, M, power):
    x = torch.randn(M, 2048, generator=torch.Generator().manual_seed(M))
    x = (x.double() * 2.0 ** -(power + torch.arange(M) % 8)[:, None]).to(torch.bfloat16).cuda()
    w, ws = weights(64, 2048)
    y, _, codes, scale, _ = ql.qlinear_int8_w8a8(x, w, ws, debug=True)
    q, s = ql.quantize_int8(x)
    assert torch.equal(q, codes) and torch.equal(s, scale)
    assert torch.equal(ql.qlinear_int8(q, s, w, ws), y)


@pytest.mark.parametrize("M,N", [(1, 64), (4, 64), (16, 64), (260, 64), (300, 6000)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_tokens_that_are_not_finite(ql, M, N, bad):
    x = torch.randn(M, 2048, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    w, ws = weights(N, 2048)
    clean = ql.qlinear_int8(*ql.quantize_int8(x), w, ws)
    at = M // 2
    x[at, 7] = bad
    y = ql.qlinear_int8(*ql.quantize_int8(x), w, ws)
    assert not y[at].isfinite().any()
    others = torch.arange(M, device="cuda") != at
    assert torch.equal(y[others], clean[others])
