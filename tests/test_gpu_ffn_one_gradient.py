"""One gradient alone needs one of x and w13: without the other the same bits come out, and what is
needed is asked for."""
import pytest
import torch

from _util import gpu_lib
from test_gpu_ffn import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("save", ["bf16", "int8"])
@pytest.mark.parametrize("M,H,I", [(1, 72, 40), (140, 264, 136)])
def test_the_operand_that_is_not_read_may_be_absent(M, H, I, save):
    ql = gpu_lib()
    x, w, dh = make(M, H, I, seed=80, pad=1)
    _, saved = ql.gated_ffn(x, w, save=save)
    dx, _ = ql.gated_ffn_backward(dh, x, w, saved, need_dw=False)
    _, dw = ql.gated_ffn_backward(dh, x, w, saved, need_dx=False)
    got, none = ql.gated_ffn_backward(dh, None, w, saved, need_dw=False)
    assert none is None and torch.equal(got, dx)
    none, got = ql.gated_ffn_backward(dh, x, None, saved, need_dx=False)
    assert none is None and torch.equal(got, dw)


def test_what_is_needed_is_asked_for():
    ql = gpu_lib()
    x, w, dh = make(40, 64, 72, seed=81)
    _, saved = ql.gated_ffn(x, w, save="int8")
    for a, b, kw in ((None, w, {}), (x, None, {}), (None, None, {}), (None, w, dict(need_dx=False)),
                     (x, None, dict(need_dw=False)), (None, None, dict(need_dx=False, need_dw=False))):
        with pytest.raises(TypeError):
            ql.gated_ffn_backward(dh, a, b, saved, **kw)
    with pytest.raises(TypeError):
        ql.gated_ffn_backward(dh, None, w.float(), saved, need_dw=False)
    with pytest.raises(TypeError):
        ql.gated_ffn_backward(dh, x.cpu(), None, saved, need_dx=False)
    with pytest.raises(TypeError):  # dh belongs to other weights
        ql.gated_ffn_backward(dh[:, :64], None, w, saved, need_dw=False)
