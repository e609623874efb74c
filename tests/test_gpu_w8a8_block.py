"""A run of the 8-bit operators together, as a W8A8 model's block uses them: tokens quantised once, their
codes through two projections, the router in bf16, the routed experts on 8-bit codes, the residual added;
for one token and a decode batch eagerly and as one captured graph, for a prompt through the projections."""
import numpy as np
import pytest
import torch

from _util import bits_of, gpu_lib
from oracle import moe_few_oracle as MO
from oracle import qlinear_oracle as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


E, TOPK, H, I = 12, 3, 512, 192


@pytest.fixture(scope="module")
def weights():
    g = torch.Generator().manual_seed(0)
    w = {n: torch.randint(-127, 128, s, generator=g, dtype=torch.int8)
         for n, s in (("mix", (H, H)), ("shared", (H, H)), ("w13", (E, 2 * I, H)), ("w2", (E, H, I)))}
    s = {n: (torch.rand(v.shape[:-1], generator=g) + 0.5) / (73 * v.shape[-1] ** 0.5) for n, v in w.items()}
    router = (torch.randn(E, H, generator=g) / H ** 0.5).to(torch.bfloat16)
    return {n: v.cuda() for n, v in w.items()}, {n: v.cuda() for n, v in s.items()}, router.cuda()


def block(ql, x, weights):
    w, s, router = weights
    codes, scale = ql.quantize_int8(x)
    mixed = ql.qlinear_int8(codes, scale, w["mix"], s["mix"])
    shared = ql.qlinear_int8(codes, scale, w["shared"], s["shared"], out_dtype=torch.float32)
    logits = ql.qlinear_bf16(mixed, router)
    y, ids, wts, h, _ = ql.moe_int8(mixed, w["w13"], s["w13"], w["w2"], s["w2"], router_logits=logits, topk=TOPK,
                                    renormalize=True, debug=True)
    return mixed, shared, logits, ids, y


@pytest.mark.parametrize("M", [1, 5, 33])
def test_block(ql, weights, M):
    w, s, router = weights
    x = torch.randn(M, H, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    mixed, shared, logits, ids, y = block(ql, x, weights)
    q, scale = ql.quantize_int8(x)
    for n, got, dtype in (("mix", mixed, torch.bfloat16), ("shared", shared, torch.float32)):
        acc = MO.linear_codes(q.cpu().numpy(), scale.cpu().numpy(), w[n].cpu().numpy(), s[n].cpu().numpy())[0]
        f = torch.from_numpy(acc.astype(np.float32) * scale.cpu().numpy()[:, None] * s[n].cpu().numpy())
        assert torch.equal(got.cpu(), f.to(dtype))
    rid, rw = Q.route_topk(bits_of(logits), TOPK, True)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # the layer on the block's own activations, in 64 bits: 8-bit h is 0.4 % of its row's largest a step, of
    # which rounding moves half at most; 2 % of y's norm is far above that and far below a wrong expert
    qm, sm = MO.codes(mixed.double().cpu().numpy())
    w13 = w["w13"].double().cpu().numpy() * s["w13"].double().cpu().numpy()[..., None]
    w2 = w["w2"].double().cpu().numpy() * s["w2"].double().cpu().numpy()[..., None]
    g, u, G, U = MO.gate_up(qm * sm, w13, rid)
    h, _ = MO.activation(g, u, 0 * G, 0 * U)
    hq, hs = MO.codes(h)
    ref, _ = MO.down(hq * hs, w2, rid, rw)
    assert np.linalg.norm(y.double().cpu().numpy() - ref) < 0.02 * np.linalg.norm(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(ql, x, weights)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, (mixed, shared, logits, ids, y)))


def test_prompt_through_the_projections(ql, weights):
    """A prompt's rows equal the same tokens' rows decoded in small batches: exact sums, one rounding."""
    w, s, _ = weights
    x = torch.randn(300, H, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    codes, scale = ql.quantize_int8(x)
    prompt = ql.qlinear_int8(codes, scale, w["mix"], s["mix"])
    for a, b in ((0, 1), (1, 12), (12, 40), (40, 300)):
        part = ql.qlinear_int8(codes[a:b].contiguous(), scale[a:b].contiguous(), w["mix"], s["mix"])
        assert torch.equal(part, prompt[a:b])
