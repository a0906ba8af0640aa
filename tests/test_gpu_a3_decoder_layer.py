"""The example decoder layer: attention operators and the MoE layer together, as a serving program runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("prompts,kw", [
    ((37, 150), {}),
    ((1, 15, 400), {"q_heads": 12, "kv_heads": 4, "head_dim": 64, "decode": 3}),
])
def test_decoding_matches_one_prefill(prompts, kw):
    """Tokens decoded one by one over the cache against the same tokens in one prefill.

    The two differ by the attention kernels' roundings (2^-8 relative), which move a few percent of the experts'
    8-bit activations by one step (2^-4): 1e-2 of a token's norm; 5e-2 is allowed.  Every expert is picked
    (top_k = experts), so that no near tie of the router can choose others."""
    assert _example().run(prompts, experts=4, top_k=4, **kw) < 5e-2
