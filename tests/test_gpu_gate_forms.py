"""The residual step's gate is told by its shape: on square inputs too, [H] is a gate for each channel, [T,1] for each token."""
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe

pytestmark = pytest.mark.gpu


def test_square_inputs():
    n = 64
    g = torch.Generator().manual_seed(0)
    x, h, dx = (torch.randn(n, n, generator=g).cuda() for _ in range(3))
    gate = torch.randn(n, generator=g).cuda()
    for form, full in ((gate, gate[None, :]), (gate[:, None], gate[:, None])):
        new, _ = moe.residual_fwd(x, h, gate=form)
        want, _ = moe.residual_fwd(x, h, gate=full.expand(n, n).contiguous())
        # x + gate h in one fused rounding, or with the product rounded first: half a step of either more
        assert ((new - want).abs() <= 2.0 ** -24 * ((form * h).abs() + new.abs() + want.abs())).all()
        d = moe.residual_bwd(new, h, dx, gate=form).d_gate
        assert d.shape == form.shape
        terms = dx.double() * h.double()
        ref = terms.sum(0) if form.dim() == 1 else terms.sum(1, keepdim=True)
        assert ((d.double() - ref).abs() <= 80 * 2.0 ** -24 * (terms.abs().sum(0) if form.dim() == 1 else terms.abs().sum(1, keepdim=True))).all()
    with pytest.raises(ValueError, match="gate"):
        moe.residual_fwd(x[:32], h[:32], gate=gate[:32])
