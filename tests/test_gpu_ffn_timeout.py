"""Waits that run out where tiles are cut along the summed dimension: the tickets are zero after every
launch, so the workspace needs no repair, and the default workspaces' status can be read.  The wait
limit of zero lets every role give up at its first unsuccessful poll; the pair then waits for its
copies in flight, frees its tensor memory and returns."""
import pytest
import torch

from _util import gpu_lib
from test_gpu_ffn import make

pytestmark = pytest.mark.gpu

SHAPES = [(40, 4096, 72), (4104, 4096, 520), (2406, 8, 1136), (6899, 784, 2352)]


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


def tickets(ws):
    return ws.buf[256:256 + (1 << 20)]


@pytest.mark.parametrize("M,H,I", SHAPES)
def test_tickets_are_whole_after_a_timeout(ql, M, H, I):
    plans = [ql.gated_ffn_plan("forward", M, I, H, save="int8"), ql.gated_ffn_plan("dx", M, I, H),
             ql.gated_ffn_plan("dw", M, I, H)]
    assert any(p.cut for p in plans)
    x, w, dh = make(M, H, I, seed=60)
    ws = ql.Workspace()

    def step():
        h, saved = ql.gated_ffn(x, w, save="int8", workspace=ws)
        return h, *ql.gated_ffn_backward(dh, x, w, saved, workspace=ws)

    want = step()
    step()
    assert ql.read_device_status(ws.buf) == (0, 0)
    seen = 0
    for limit in (0, 0, 0, 0, 1, 2, 4, 8, 16, 32, 64, 128):  # some calls lose all parts, some a few
        ql.set_wait_limit(limit)
        try:
            step()
        finally:
            ql.set_wait_limit(1 << 20)
        st, flags = ql.read_device_status(ws.buf, clear=True)
        seen += flags & 1
        assert not bool(tickets(ws).any())
        got = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert ql.read_device_status(ws.buf) == (0, 0)
    assert seen


def test_default_workspaces_tell_and_recover(ql):
    M, H, I = SHAPES[0]
    x, w, dh = make(M, H, I, seed=61)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        want = ql.gated_ffn(x, w, save="bf16")[0]
    ql.read_device_status()  # whatever earlier tests left
    assert ql.read_device_status() == (0, 0)
    ql.set_wait_limit(0)
    try:
        for _ in range(8):
            with torch.cuda.stream(st):
                ql.gated_ffn(x, w, save="bf16")
            status, flags = ql.read_device_status()
            if flags & 1:
                break
    finally:
        ql.set_wait_limit(1 << 20)
    assert status != 0 and flags & 1
    assert ql.read_device_status() == (0, 0)
    with torch.cuda.stream(st):
        got = ql.gated_ffn(x, w, save="bf16")[0]
    st.synchronize()
    assert torch.equal(got, want)
