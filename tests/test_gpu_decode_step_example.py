"""The decode-step example: weights, cache and shared-prefix attention as a program uses them together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("args", [[], ["--cache", "q4_0", "--batch", "3", "--prompt", "77", "--steps", "2"],
                                  ["--batch", "5", "--prompt", "1", "--steps", "70"]])
def test_decode_step_example(args):
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.main(args)  # raises if the attention is off its definition, or anything was recorded
