"""The gated block's workspaces under CUDA graphs: graphs captured with the default workspaces are
independent of each other and of later calls, and a workspace that a graph was captured with outlives
its replacement by a larger one.  The shapes cut tiles along the summed dimension, so that a call
counts on tickets that are zero."""
import pytest
import torch

from _util import gpu_lib
from test_gpu_ffn import make

pytestmark = pytest.mark.gpu

SHAPES = [(40, 4096, 72), (2406, 8, 1136)]  # the forward's tiles are cut; both gradients' are


@pytest.fixture(scope="module")
def ql():
    return gpu_lib()


def step(ql, t, **kw):
    x, w, dh = t
    h, saved = ql.gated_ffn(x, w, save="int8", **kw)
    dx, dw = ql.gated_ffn_backward(dh, x, w, saved, **kw)
    return h, dx, dw


def same(a, b):
    return all(torch.equal(i, j) for i, j in zip(a, b))


@pytest.fixture(scope="module")
def cases(ql):
    M, H, I = SHAPES[0]
    assert ql.gated_ffn_plan("forward", M, I, H, save="int8").cut
    M, H, I = SHAPES[1]
    assert ql.gated_ffn_plan("dx", M, I, H).cut and ql.gated_ffn_plan("dw", M, I, H).cut
    sets = [make(*s, seed=30 + i) for i, s in enumerate(SHAPES + SHAPES)]
    want = [step(ql, t) for t in sets]
    torch.cuda.synchronize()
    return sets, want


def capture(f):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    return g, out


def test_captures_leave_no_default_workspace_behind(ql, cases):
    sets, _ = cases
    before = {k: w.buf.data_ptr() for k, w in ql._ffn_workspaces.items()}
    graphs = [capture(lambda: step(ql, t)) for t in sets]
    assert {k: w.buf.data_ptr() for k, w in ql._ffn_workspaces.items()} == before
    del graphs


def test_graphs_in_reverse_order_and_on_two_streams(ql, cases):
    sets, want = cases
    graphs = [capture(lambda: step(ql, t)) for t in sets]
    for g, out in reversed(graphs):
        g.replay()
    torch.cuda.synchronize()
    for (_, out), ref in zip(graphs, want):
        assert same(out, ref)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_, out), ref in zip(graphs, want):
        assert same(out, ref)


def test_default_calls_between_replays(ql, cases):
    """Eager calls of a larger size on the capturing stream replace its default workspace; the graph
    holds none of it."""
    sets, want = cases
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step(ql, sets[0])
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        out = step(ql, sets[0])
    with torch.cuda.stream(st):
        assert same(step(ql, sets[1]), want[1])
        filler = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
        g.replay()
    torch.cuda.synchronize()
    assert same(out, want[0]) and all(bool((f == 7).all()) for f in filler)


def test_a_recorded_workspace_is_not_freed(ql, cases):
    sets, want = cases
    ws = ql.Workspace()
    step(ql, sets[0], workspace=ws)
    # the forward comes first and needs the most: one buffer from here on
    size, at = ws.buf.numel(), ws.buf.data_ptr()
    torch.cuda.synchronize()
    g, out = capture(lambda: step(ql, sets[0], workspace=ws))
    assert ws.buf.data_ptr() == at
    big = make(3000, 512, 2048, seed=40)
    step(ql, big, workspace=ws)
    assert ws.buf.numel() > size
    filler = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert same(out, want[0]) and all(bool((f == 7).all()) for f in filler)


def test_a_workspace_too_small_for_the_capture_is_left_alone(ql, cases):
    sets, want = cases
    ws = ql.Workspace()
    g, out = capture(lambda: step(ql, sets[1], workspace=ws))
    assert ws.buf is None
    assert same(step(ql, sets[1], workspace=ws), want[1])  # before the graph has run once
    g.replay()
    torch.cuda.synchronize()
    assert same(out, want[1])


def test_one_gradient_and_few_tokens_captured(ql, cases):
    """Calls that count on no tickets zero none: they are right in memory that holds anything."""
    sets, want = cases
    x, w, dh = sets[1]
    _, saved = ql.gated_ffn(x, w, save="int8")
    dx, _ = ql.gated_ffn_backward(dh, x, w, saved, need_dw=False)
    h = ql.gated_ffn(x[:4], w)
    g, out = capture(lambda: (ql.gated_ffn_backward(dh, x, w, saved, need_dw=False)[0], ql.gated_ffn(x[:4], w)))
    g.replay()
    torch.cuda.synchronize()
    assert same(out, (dx, h))


def test_many_calls_in_one_graph_share_its_workspace(ql, cases):
    """Sizes that grow and shrink, replayed twice: the second replay finds what the first left."""
    sets, want = cases
    order = [0, 1, 0, 3, 2, 1]
    g, out = capture(lambda: [step(ql, sets[i]) for i in order])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for got, i in zip(out, order):
        assert same(got, want[i])


def test_eager_calls_while_another_stream_is_captured(ql, cases):
    sets, want = cases
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(ql, sets[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        first = step(ql, sets[1])
        with torch.cuda.stream(side):
            eager = step(ql, sets[1])
        second = step(ql, sets[3])
    step(ql, sets[0])
    assert not ql._ffn_captures
    g.replay()
    torch.cuda.synchronize()
    assert same(first, want[1]) and same(second, want[3]) and same(eager, want[1])


def test_branches_of_a_graph_do_not_share(ql, cases):
    """Calls on two streams of one capture run side by side when it is replayed."""
    sets, want = cases
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            b = [step(ql, sets[3]) for _ in range(4)]
        a = [step(ql, sets[1]) for _ in range(4)]
        main.wait_stream(side)
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert all(same(t, want[1]) for t in a) and all(same(t, want[3]) for t in b)
