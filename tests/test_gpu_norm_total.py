"""Norms whose result takes x's place, without a residual: what is returned for the total."""
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq

pytestmark = pytest.mark.gpu
KINDS = [(1, 64), (5, 96), (7, 1999), (2, 40000), (900, 1024)]


@pytest.mark.parametrize("rows,D", KINDS)
def test_in_place_without_a_residual(rows, D):
    """y in x's place leaves no total: None is returned for it, and the gradient refuses that instead of taking y for it."""
    x, w = torch.randn(rows, D, device="cuda"), torch.randn(D, device="cuda")
    y, total, rstd = pnq.rms_norm(x, w)
    assert total is x
    codes, scales, total = pnq.rms_norm_int8(x, w, y=torch.empty_like(x))
    assert total is x
    for held in (x.clone(), x.clone()[:, :]):
        got, total, r = pnq.rms_norm(held, w, out=held)
        assert got is held and total is None and torch.equal(got, y) and torch.equal(r, rstd)
        with pytest.raises(TypeError, match="total"):
            pnq.rms_norm_backward(y, total, w, r)
    held = x.clone()
    assert pnq.rms_norm(held, w, out=held.view(rows, D))[1] is None  # another tensor of the same memory
    held = x.clone()
    c, s, total = pnq.rms_norm_int8(held, w, y=held)
    assert total is None and torch.equal(held, y) and torch.equal(c, codes) and torch.equal(s, scales)
