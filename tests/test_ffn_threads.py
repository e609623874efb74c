"""Host threads that call the gated block on one stream (no GPU: the library and the tensors are fakes).
A call's launches hand [dg du] on in the workspace, so no two calls may be inside the library with the
same workspace at once; the buffer must not be replaced meanwhile either."""
import threading
import time

import pytest
import torch

from _util import gpu_lib


class Fake:
    """As much of a CUDA tensor as the binding looks at."""
    device, is_cuda = torch.device("cuda", 0), True

    def __init__(self, shape, dtype=torch.bfloat16, at=4096):
        self.shape, self.dtype, self.at = tuple(shape), dtype, at

    def stride(self, i=None):
        s, n = [], 1
        for d in reversed(self.shape):
            s.insert(0, n)
            n *= d
        return tuple(s) if i is None else s[i]

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.shape[0]

    def is_contiguous(self):
        return True


class Library:
    """Counts the calls that are inside with the same workspace; each stays for a while."""

    def __init__(self, real):
        self.real, self.inside, self.worst, self.guard = real, {}, 0, threading.Lock()

    def __getattr__(self, name):
        return getattr(self.real, name)

    def ql_workspace_init(self, *a):
        return 0

    def ql_capture_id(self, stream):
        return 0

    def gated_ffn(self, *a):
        return self.call(a[14])

    def gated_ffn_backward(self, *a):
        return self.call(a[18])

    def call(self, ws):
        with self.guard:
            self.inside[ws] = self.inside.get(ws, 0) + 1
            self.worst = max(self.worst, self.inside[ws])
        time.sleep(0.02)
        with self.guard:
            self.inside[ws] -= 1
        return 0


@pytest.fixture
def ql(monkeypatch):
    ql = gpu_lib()
    monkeypatch.setattr(ql, "lib", Library(ql.lib))
    monkeypatch.setattr(ql, "_stream", lambda stream=None: 5)
    monkeypatch.setattr(ql, "_ffn_workspaces", {})
    at = iter(range(1 << 20, 1 << 40, 1 << 20))
    monkeypatch.setattr(torch, "empty", lambda n, **kw: Fake((n,), torch.uint8, next(at)))
    return ql


def both_ways(ql, M, **kw):
    H, I = 64, 128
    x, w, dh, h = Fake((M, H)), Fake((2 * I, H)), Fake((M, I)), Fake((M, I))
    saved = ql.FFNCheckpoint("int8", Fake((M, 2, 128), torch.int8), Fake((M, 2, 1), torch.float32))
    ql.gated_ffn(x, w, out=h, **kw)
    ql.gated_ffn_backward(dh, x, w, saved, out_dx=Fake((M, H)), out_dw=Fake((2 * I, H)), **kw)


@pytest.mark.parametrize("given", [False, True])
def test_calls_with_one_workspace_follow_each_other(ql, given):
    kw = dict(workspace=ql.Workspace("cuda:0")) if given else {}
    errors = []

    def run(M):
        try:
            for _ in range(3):
                both_ways(ql, M, **kw)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(40 + 8 * i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and ql.lib.worst == 1


def test_the_lock_is_free_after_a_refusal(ql, monkeypatch):
    ws = ql.Workspace("cuda:0")
    monkeypatch.setattr(ql.lib, "call", lambda at: 4, raising=False)
    with pytest.raises(ql.QLError):
        both_ways(ql, 40, workspace=ws)
    assert not ws.lock.locked()

    def no_memory(n, **kw):
        raise MemoryError

    monkeypatch.setattr(torch, "empty", no_memory)
    with pytest.raises(MemoryError):
        both_ways(ql, 40, workspace=ql.Workspace("cuda:0"))
    ws.buf = None
    with pytest.raises(MemoryError):
        both_ways(ql, 40, workspace=ws)
    assert not ws.lock.locked()
