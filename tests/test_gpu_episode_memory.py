"""The sequence memory in use: examples/episode_memory.py trains and acts."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_trains_and_acts():
    spec = importlib.util.spec_from_file_location("episode_memory", os.path.join(ROOT, "examples", "episode_memory.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, acted, read, right, status = ex.main(steps=60, n=48, length=100, say=lambda s: None)
    assert status == {"bad_index": 0, "timeout": 0}
    # the value of an episode that forgot its sign is zero: loss 0.5
    assert losses[0] > 0.4 and sum(losses[-5:]) / 5 < 0.2
    assert right >= 0.95
    # both round each output to bf16 once, and the chunked pass its operands to 11 bits: outputs agree within
    # 2^-8 of their size and a value, about one in size, is a sum of 128 of them with errors of either sign
    assert (acted - read).abs().max().item() < 2.0 ** -4
