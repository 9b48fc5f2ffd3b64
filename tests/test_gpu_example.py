"""The example layer, end to end."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "moe_decoder.py")


@pytest.mark.parametrize("tokens,d,hidden,experts,topk", [(1, 256, 128, 8, 2), (7, 512, 384, 16, 4), (40, 1024, 512, 8, 2)])
def test_layer(tokens, d, hidden, experts, topk):
    spec = importlib.util.spec_from_file_location("moe_decoder", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    print("example", tokens, d, hidden, experts, topk, flush=True)
    stream, y, losses = example.run(tokens, d, hidden, experts, topk)
    # E4M3 rounds an element by at most 2^-4 of it, 2^-4 / sqrt(3) in the root mean square.  The stream
    # takes one such rounding (of the projection's operand) and three roundings to bf16; the experts'
    # output takes that one twice (gate and up), its own operand's twice and the hidden rows' once.
    rounding = 2.0 ** -4 / 3 ** 0.5
    assert stream < rounding + 3 * 2.0 ** -8
    assert y < 5 * rounding + 4 * 2.0 ** -8
    # half of the way to the target each step: a quarter of the loss, down to the rounding's share
    assert all(b < 0.5 * a for a, b in zip(losses[:3], losses[1:4]))
    assert losses[-1] < losses[0] / 16
