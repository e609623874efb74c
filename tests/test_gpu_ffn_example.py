"""The example that trains the gated block, quantises it and decodes with it, end to end."""
import importlib.util
import os

import pytest

from _util import ROOT, gpu_lib

pytestmark = pytest.mark.gpu


def test_train_quantise_decode():
    gpu_lib()
    spec = importlib.util.spec_from_file_location("example", os.path.join(ROOT, "examples", "gated_ffn_train_then_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    first, last, off = m.main(60)
    assert last < 0.5 * first
    # 4-bit rounding of both weights: a step of a 16th of a group's range, about 0.1 of a normal weight
    assert off < 0.3
