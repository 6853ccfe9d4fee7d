"""Calls at the edges of the decoder operators, on the GPU: what is not finite beside what is, values at the end of a type's range,
caches and lists far longer than those of tests/test_gpu_decoder.py, streams and graphs of their own."""
import pytest
import torch

import nvfp4_block_scaled_elem_amd as nv
from tests import decoder_ref as dref
from tests import test_gpu_moe as moe_of

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def say(msg):
    print(msg, flush=True)


# ------------------------------------------------------------------------------------------- experts

@pytest.mark.parametrize("tokens", [2, 3, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("which", ["up", "down"])
@pytest.mark.parametrize("bad", ["scale", "alpha"])
def test_weights_that_are_not_finite_stay_with_their_tokens(tokens, which, bad):
    """A NaN scale byte or an infinite alpha of an expert reaches the tokens that chose it, and no others: they are what they
    are with sound weights, bit for bit."""
    say(f"not finite weights {tokens} {which} {bad}")
    up, down = moe_of.layer(1, 8, 256, 160, True)
    x, logits = moe_of.rand(1, tokens, 256), moe_of.rand(2, tokens, 8, dtype=F32)
    logits[0, 5], logits[1, 5] = 30.0, -30.0  # chosen by the first, not by the second
    clean = nv.moe(x, logits, up, down, 2)
    chosen, _, _ = dref.route(logits, 2, False, True)
    W = up if which == "up" else down
    if bad == "scale":
        W[1][5] = 0x7F
    else:
        W[2][5] = float("inf")
    y = nv.moe(x, logits, up, down, 2)
    mine = chosen[:, 5]
    assert mine[0] and not mine[1]
    assert not torch.isfinite(y[mine]).any() if bad == "scale" else not torch.isfinite(y[mine]).all()
    assert torch.equal(y[~mine], clean[~mine])
