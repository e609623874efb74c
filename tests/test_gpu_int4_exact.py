"""Long sums of the 4-bit linear, exactly.  A bound of K 2^-23 sum|x w| is too wide at K = 17408 to see a
lost piece of K; here the activations are whole numbers in -3..3, the zero points 0..15 and the scales
powers of two, so that every sum is a multiple of 2^-3 below 2^21: fp32 holds it whatever the order,
and every output has to be the rounded sum bit for bit.

One token's activations are staged for a CTA 32 KB at a time (96 blocks of 128 k; 128 with groups
shorter than 128) where its share of K is longer: 9760 rows and K = 17408 are 305 row tiles, enough
that K is not shared by a cluster, so a CTA stages 136 blocks in two pieces, the second of 40 or of 8
blocks; 19457 rows and more go to the form with four row groups."""
import pytest
import torch

from _util import gpu_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


def make(M, N, K, group, zeros, dtype, down=0):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, device="cuda", generator=g)

    groups = -(-K // group)
    x = ints(-3, 4, M, K).to(torch.bfloat16)
    w = ints(0, 256, N, K // 2).to(torch.uint8)
    s = (2.0 ** (ints(-3, 1, N, groups) - down)).to(dtype)
    return x, w, s, ints(0, 16, N, groups).to(torch.uint8) if zeros else None


def sums(x, w, s, z, group, step=2048):
    """In 64 bits, some rows of W at a time."""
    K = x.shape[1]
    at = torch.arange(K, device=w.device) // group
    out = []
    for i in range(0, w.shape[0], step):
        r = slice(i, i + step)
        q = torch.stack((w[r] & 15, w[r] >> 4), 2).reshape(-1, K).double()
        zero = 8.0 if z is None else z[r].double()[:, at]
        out.append(x.double() @ ((q - zero) * s[r].double()[:, at]).t())
    return torch.cat(out, 1)


def check(ql, M, N, K, group, zeros, dtype):
    x, w, s, z = make(M, N, K, group, zeros, dtype)
    want = sums(x, w, s, z, group)
    assert float(want.abs().max()) < 2.0 ** 21
    assert torch.equal(ql.qlinear_int4(x, w, s, z, group=group), want.float().to(torch.bfloat16))


FORMS = [(32, True, torch.bfloat16), (64, False, torch.float16), (128, True, torch.float16),
         (128, False, torch.bfloat16), (512, True, torch.bfloat16), (1 << 20, False, torch.float16)]


# few rows (K over a CTA's warps and a cluster's CTAs), rows for two CTAs per SM, K that ends inside a
# block of 128, and each number of tokens that a launch takes
@pytest.mark.parametrize("group,zeros,dtype", FORMS)
@pytest.mark.parametrize("M", [1, 2, 8, 9, 16, 17, 32, 45])
@pytest.mark.parametrize("N,K", [(96, 17408), (640, 17376), (5000, 17312)])
def test_long_sums(ql, M, N, K, group, zeros, dtype):
    check(ql, M, N, K, group, zeros, dtype)


@pytest.mark.parametrize("group,zeros,dtype", FORMS)
@pytest.mark.parametrize("N,K", [(9760, 17408), (9761, 17312), (9760, 12320), (14592, 17408), (14593, 17376), (19500, 17408), (19457, 25632), (19500, 16416)])
def test_one_token_staged_in_pieces(ql, N, K, group, zeros, dtype):
    check(ql, 1, N, K, group, zeros, dtype)


@pytest.mark.parametrize("group,zeros,dtype", FORMS)
@pytest.mark.parametrize("M,I,H", [(1, 4904, 17408), (1, 9752, 17312), (1, 40, 17408), (6, 1032, 8224), (30, 264, 17376)])
def test_gated_long_sums(ql, M, I, H, group, zeros, dtype):
    """g and u are exact, so the block's output is that of the bf16 block on the same weights (whose g and
    u are exact too), bit for bit."""
    x, w, s, z = make(M, 2 * I, H, group, zeros, dtype, down=10)
    at = torch.arange(H, device="cuda") // group
    wide = torch.empty(2 * I, H, dtype=torch.bfloat16, device="cuda")
    for i in range(0, 2 * I, 2048):
        r = slice(i, i + 2048)
        q = torch.stack((w[r] & 15, w[r] >> 4), 2).reshape(-1, H).float()
        wide[r] = ((q - (8.0 if z is None else z[r].float()[:, at])) * s[r].float()[:, at]).to(torch.bfloat16)
    got, path = ql.gated_ffn_int4(x, w, s, z, group=group, swiglu_alpha=1.25, swiglu_limit=3.0, debug=True)
    assert path == "gated_ffn_int4"
    assert torch.equal(got, ql.gated_ffn(x, wide, swiglu_alpha=1.25, swiglu_limit=3.0))
