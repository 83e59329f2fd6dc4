"""The FP8 expert-layer example: one call and its operators agree, a captured step gives the eager step's bits."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("args", [[], ["--tokens", "5", "--hidden", "400", "--inter", "208", "--experts", "12", "--top-k", "3"]])
def test_example(args):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_expert_layers.py")
    spec = importlib.util.spec_from_file_location("fp8_expert_layers", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    apart, same = mod.main(args)
    # the sum with the shared row, some three times the routed sum's size, is rounded to bf16 (2^-9.2 rms
    # of it, 2^-7.6 of the routed sum), the other by itself, and codes turn as in the layer's tests (2^-7)
    assert apart < 2.0 ** -6 and same
