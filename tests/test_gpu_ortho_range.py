"""Orthogonalisation at the ends of the range: the norm and eps are sums and doubles, their quotient must not be lost."""
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe

pytestmark = pytest.mark.gpu


def updates(M, N, dtype=torch.float32):
    return torch.randn(3, M, N, generator=torch.Generator().manual_seed(M)).to(dtype).cuda()


@pytest.mark.parametrize("M,N", [(72, 136), (136, 72)])
def test_infinite_eps_gives_zero(M, N):
    """U / (|U| + inf) = 0, and zero stays zero."""
    for dtype in (torch.float32, torch.bfloat16):
        o, _ = moe.orthogonalize(updates(M, N, dtype), eps=float("inf"), dtype="fp32")
        assert not o.any()


@pytest.mark.parametrize("eps", [1e-7, 0.0, float("inf")])
@pytest.mark.parametrize("steps", [1, 2, 5])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("M,N", [(72, 136), (136, 72), (8, 264)])
def test_non_finite_element_makes_its_matrix_nan(M, N, value, steps, eps):
    u = updates(M, N)
    want, _ = moe.orthogonalize(u, steps=steps, eps=eps)
    u[1, M // 2, N // 3] = value
    got, _ = moe.orthogonalize(u, steps=steps, eps=eps)
    assert torch.isnan(got[1]).all() and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("power", [-126, -60, 60, 120])
@pytest.mark.parametrize("M,N", [(72, 136), (136, 72)])
def test_a_power_of_two_changes_nothing(M, N, power):
    """Without eps X does not depend on the update's size: at most the last bits of the two factors."""
    u = updates(M, N)
    a, _ = moe.orthogonalize(u, eps=0.0, dtype="fp32")
    b, _ = moe.orthogonalize(u * 2.0 ** power, eps=0.0, dtype="fp32")
    assert (a.double() - b.double()).norm() <= 2.0 ** -9 * a.double().norm()   # as far as two results of one update may be
