"""Edges of the mixture-of-experts layers for a few tokens: what the debug output holds for padding."""
import numpy as np
import pytest
import torch

from _util import gpu_lib
from test_gpu_moe_few import Layer, check, tokens

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
