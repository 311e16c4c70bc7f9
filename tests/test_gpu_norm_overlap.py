"""Norms whose result takes an operand's place: as apart from them, or refused."""
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq

pytestmark = pytest.mark.gpu
KINDS = [(1, 64), (5, 96), (7, 1999), (2, 40000), (900, 1024)]


@pytest.mark.parametrize("rows,D", KINDS)
def test_in_place_with_a_residual(rows, D):
    """y in x's or the residual's place, the total in the other's: the same as apart."""
    x, res, w = torch.randn(rows, D, device="cuda"), torch.randn(rows, D, device="cuda"), torch.randn(D, device="cuda")
    y, total, rstd = pnq.rms_norm(x, w, residual=res)
    for place in ("y in x", "y in residual", "crossed"):
        a, b = x.clone(), res.clone()
        kw = {"y in x": dict(out=a, total=b), "y in residual": dict(out=b), "crossed": dict(out=b, total=a)}[place]
        got = pnq.rms_norm(a, w, residual=b, **kw)
        assert all(torch.equal(g, v) for g, v in zip(got, (y, total, rstd))), place


def test_overlaps_are_refused():
    rows, D = 4, 64
    buf, w, rstd = torch.randn(4 * rows * D, device="cuda"), torch.randn(D, device="cuda"), torch.rand(rows, device="cuda")
    at = lambda first: buf[first: first + rows * D].view(rows, D)  # noqa: E731
    x, res = at(0), at(rows * D)
    before = buf.clone()
    for call in (lambda: pnq.rms_norm(x, w, out=at(D)), lambda: pnq.rms_norm(x, w, residual=res, total=at(rows * D - 1)),
                 lambda: pnq.rms_norm(x, w, residual=res, out=at(2 * rows * D), total=at(2 * rows * D)),
                 lambda: pnq.rms_norm(buf.view(8, 2 * D)[:rows, :D], w, out=at(0)),
                 lambda: pnq.rms_norm_int8(x, w, residual=res, y=at(2 * rows * D), total=at(2 * rows * D + 1)),
                 lambda: pnq.rms_norm_backward(x, res, w, rstd, out=at(1)), lambda: pnq.rms_norm_backward(x, res, w, rstd, out=at(rows * D)),
                 lambda: pnq.rms_norm_backward(x, res, w, rstd, at(2 * rows * D), out=at(2 * rows * D + D)),
                 lambda: pnq.expert_route_backward(torch.zeros(rows, 2, device="cuda"), x, torch.zeros(rows, 2, dtype=torch.int32, device="cuda"), out=at(D))):
        with pytest.raises(pnq.PnqError) as e:
            call()
        assert e.value.status == pnq.Status.ERR_VALUE
    assert torch.equal(buf, before)


def test_between_the_rows():
    """A result between the rows of a strided operand shares nothing with them."""
    buf = torch.randn(3, 512, device="cuda")
    x, w = buf[:, :64], torch.randn(64, device="cuda")
    out = buf[1, 128:128 + 192].view(3, 64)
    want = pnq.rms_norm(x.contiguous(), w)[0]
    y, total, _ = pnq.rms_norm(x, w, out=out)
    assert torch.equal(y, want) and total is x
