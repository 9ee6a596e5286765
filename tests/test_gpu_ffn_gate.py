"""The feed-forward block's gradient with respect to its gate, token by token, at logits where s (1 - s) is small.

s (1 - s) = t / (1 + t)^2 with t = exp(-|logit|): exp is off by two fp32 roundings, the sum, square and quotient by one
each, the product with <r, a> by one more, so that d_gate keeps its relative accuracy at any logit.  <r, a> has the bound
of the other tests: fp32 sums over H and I, phi's from the gate and up values'."""
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
from tests._block import E, SECOND, Ffn

pytestmark = pytest.mark.gpu
LOGITS = [-80.0, -60.0, -30.0, -20.0, -16.0, -12.0, -10.0, -4.0, -0.5, 0.0, 0.5, 4.0, 10.0, 12.0, 16.0, 17.5, 20.0, 30.0, 60.0, 80.0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("saved", [True, False])
@pytest.mark.parametrize("H,I", [(136, 72), (72, 264)])
def test_any_logit(H, I, saved, dtype):
    g = torch.Generator().manual_seed(H)
    rand = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(dtype).cuda()  # noqa: E731
    T = 3 * len(LOGITS) + 1
    x, gu, dn, dout = rand(T, H), rand(2 * I, H, std=H ** -0.5), rand(H, I, std=I ** -0.5), rand(T, H)
    gate = torch.tensor((LOGITS * 4)[:T], device="cuda")
    kept = moe.ffn_fwd(x, gu, dn, gate=gate, save=True)[1] if saved else None
    _, got, _, _, _ = moe.ffn_bwd(x, gu, dn, dout, gate=gate, saved=kept)
    ref = Ffn(x, gu, dn, "swiglu", "concat", gate)
    r = dout.double() @ ref.dn
    er = H * E * (dout.double().abs() @ ref.dn.abs())
    t = torch.exp(-gate.double().abs())
    slope = t / (1 + t) ** 2
    ra = r * ref.a
    err = (er * ref.a.abs() + r.abs() * ref.ea + (I + 8) * E * ra.abs()).sum(1) + 6 * E * ra.sum(1).abs()
    want = slope * ra.sum(1)
    over = (got.double() - want).abs() - SECOND * slope * err
    assert over.max().item() <= 0, (gate[over.argmax()].item(), got[over.argmax()].item(), want[over.argmax()].item())
