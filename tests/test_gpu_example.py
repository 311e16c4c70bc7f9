"""The expert layer example on the GPU: every operator of the layer together, against the layer in 64 bits on the decoded
values. Bound: bf16 rows and results (2^-8 each: the first product, the gate, the second product, the combine; four
of them add to at most 4 * 2^-8 of the norm, and an encoded gate value that falls to the other side of a code for a
rounding of its input moves by a sixth of its group's largest at most, for a few in a thousand)."""
import os
import sys

import pytest

import block_quantized_weight_pn3t_gb300 as pnq

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("kind", [pnq.NVFP4, pnq.MXFP4])
@pytest.mark.parametrize("tokens,experts,slots,hidden,inner", [(1, 8, 2, 256, 128), (37, 16, 4, 512, 352), (700, 8, 2, 1024, 768)])
def test_expert_layer(kind, tokens, experts, slots, hidden, inner):
    import expert_layer
    err, whole, dweights = expert_layer.run(tokens, experts, slots, hidden, inner, kind)
    assert err <= 4 * 2.0 ** -8 + 0.01
    assert whole <= 3 * 2.0 ** -8  # bf16: the scaled rows, their sum, and weights whose sum is 1 up to fp32
    assert dweights.shape == (tokens, slots) and bool(dweights.isfinite().all())
