"""The 64-bit definitions of the few-token expert layers and the 8-bit-code linear, pinned by hand and by
other formulas."""
import numpy as np
import torch

from oracle import moe_few_oracle as MO


def test_codes_by_hand():
    q, s = MO.codes(np.array([[12.7, -6.35, 0.05, 0.0], [0.0, 0.0, 0.0, 0.0], [254.0, 1.0, 3.0, -5.0]]))
    assert np.allclose(s[:, 0], [0.1, 0.0, 2.0])
    assert np.array_equal(q[1], [0, 0, 0, 0])
    assert np.array_equal(q[2], [127, 0, 2, -2])  # .5, 1.5, -2.5: to even
    assert q[0, 0] == 127 and q[0, 3] == 0


def test_layer_is_the_sum_over_experts():
    g = np.random.default_rng(0)
    E, I, H, M, topk = 5, 6, 8, 3, 2
    w13, w2, x = g.standard_normal((E, 2 * I, H)), g.standard_normal((E, H, I)), g.standard_normal((M, H))
    ids = np.array([[4, 0], [2, -1], [3, 3]])
    wt = g.random((M, topk))
    gt, u, G, U = MO.gate_up(x, w13, ids)
    h, off = MO.activation(gt, u, 0 * G, 0 * U, alpha=1.2, limit=0.7)
    y, a = MO.down(h, w2, ids, wt)
    want = torch.zeros(M, H, dtype=torch.float64)
    for m in range(M):
        for j in range(topk):
            e = ids[m, j]
            if e < 0:
                continue
            p = torch.from_numpy(w13[e]) @ torch.from_numpy(x[m])
            gate, up = p[:I].clamp(max=0.7), p[I:].clamp(-0.7, 0.7)
            want[m] += wt[m, j] * (torch.from_numpy(w2[e]) @ (torch.nn.functional.silu(1.2 * gate) * up))
    assert np.allclose(y, want.numpy(), rtol=1e-12, atol=1e-13)
    assert (a >= np.abs(y) - 1e-12).all() and (off >= 0).all()
    assert not gt[3].any() and not h[3].any()


def test_a_planted_mistake_shows():
    g = np.random.default_rng(1)
    w13, x, ids = g.standard_normal((2, 8, 16)), g.standard_normal((1, 16)), np.array([[1]])
    gt, u, G, U = MO.gate_up(x, w13, ids)
    h, off = MO.activation(gt, u, 2.0 ** -20 * G, 2.0 ** -20 * U)
    swapped, _ = MO.activation(u, gt, 0 * G, 0 * U)
    assert (np.abs(swapped - h) > off).any()


def test_linear_codes_by_hand():
    acc, y = MO.linear_codes(np.array([[127, -128]], np.int8), np.array([0.5], np.float32),
                             np.array([[-128, -128], [1, 0]], np.int8), np.array([2.0, 0.25], np.float32))
    assert acc.tolist() == [[127 * -128 + 128 * 128, 127]] and y.tolist() == [[128.0, 15.875]]
