"""One workspace for the few-token mixture-of-experts layers, the linear on 8-bit codes, the gated block and the
library's other layers in turn: every result is that of the same call on a workspace of its own, and what is zero
between calls is."""
import pytest
import torch

from _util import gpu_lib
from test_gpu_moe_few import Layer, tokens
from test_gpu_workspace_sharing import _calls

pytestmark = pytest.mark.gpu

ZERO = slice(256, 256 + (1 << 20))  # tickets, maxima and cells


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


def new_calls(ql):
    def moe(fmt, M, E, H, I):
        layer = Layer(fmt, E, H, I, seed=M)
        x = tokens(M, H, seed=M, fmt=fmt)
        logits = torch.randn(M, E, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
        return f"moe_{fmt} {M}", lambda ws: layer(ql, x, router_logits=logits, topk=3, workspace=ws)

    def codes(M, N, K):
        g = torch.Generator().manual_seed(M)
        x, w = (torch.randint(-128, 128, s, generator=g, dtype=torch.int8).cuda() for s in ((M, K), (N, K)))
        xs, ws = torch.rand(M, generator=g).cuda(), torch.rand(N, generator=g).cuda()
        return f"codes {M}", lambda space: ql.qlinear_int8(x, xs, w, ws, out_dtype=torch.float32, workspace=space)

    def gated(M):
        g = torch.Generator().manual_seed(M)
        x, w13, dh = (torch.randn(s, generator=g).to(torch.bfloat16).cuda() for s in ((M, 512), (528, 512), (M, 264)))

        def call(ws):
            h, saved = ql.gated_ffn(x, w13, save="bf16", workspace=ws)
            return torch.cat((h.flatten(), *(d.flatten() for d in ql.gated_ffn_backward(dh, x, w13, saved, workspace=ws))))
        return f"gated {M}", call

    return [moe("int8", 1, 8, 512, 256), codes(4, 640, 1024), moe("int4", 9, 5, 288, 160), moe("int8", 40, 6, 2080, 96),
            codes(30, 6016, 4112), moe("bf16", 3, 9, 520, 264), gated(150), codes(300, 1000, 1040), moe("int8", 5, 3, 96, 64)]


def test_interleaved_with_the_other_layers(ql):
    old, new = _calls(ql), new_calls(ql)
    order = []
    for i in range(max(len(old), len(new))):
        order += new[i:i + 1] + old[i:i + 1]
    order += order[::-1]
    shared = ql.Workspace()
    shared.get(64 << 20)  # sized once, so that no call gets a freshly zeroed buffer
    assert all(ql.workspace_bytes(ql.OP_INT8_CODES, *s) < 64 << 20 for s in ((300, 1000, 1040), (30, 6016, 4112)))
    fresh = {}
    for name, f in order:
        if name not in fresh:
            fresh[name] = f(ql.Workspace())
            torch.cuda.synchronize()
    for name, f in order:
        got = f(shared)
        torch.cuda.synchronize()
        assert torch.equal(got, fresh[name]), f"{name}: result differs on the shared workspace"
        assert not shared.buf[ZERO].any(), f"{name}: left something where zeros are expected"
    assert shared.buf.numel() == 64 << 20
    assert ql.read_device_status(shared.buf) == (0, 0)
