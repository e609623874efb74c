"""Backward passes of several host threads on one stream, with the default workspace."""
import threading

import pytest
import torch

from _util import gpu_lib
from test_gpu_ffn import make

pytestmark = pytest.mark.gpu


def test_threads_on_one_stream():
    ql = gpu_lib()
    sets = [make(300 + 40 * i, 512, 264, seed=50 + i) for i in range(4)]
    saved = [ql.gated_ffn(x, w, save="int8")[1] for x, w, _ in sets]
    want = [ql.gated_ffn_backward(dh, x, w, s) for (x, w, dh), s in zip(sets, saved)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    start, wrong = threading.Barrier(len(sets)), []

    def run(i):
        x, w, dh = sets[i]
        with torch.cuda.stream(st):
            start.wait(30)
            got = [ql.gated_ffn_backward(dh, x, w, saved[i]) for _ in range(50)]
        st.synchronize()
        if not all(torch.equal(a, want[i][0]) and torch.equal(b, want[i][1]) for a, b in got):
            wrong.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
