"""Every instance of every dense product against 64 bits: the feed-forward block and the orthogonalisation on each of
their tiles, with rows, columns and k past the last whole tile (tests/test_tile_coverage.py holds the shapes to that)."""
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
from tests._block import half_step, newton_schulz
from tests._tiles import FFN_SHAPES, FFN_VARIANTS, STACKS
from tests.test_gpu_ffn import inputs, run
from tests.test_gpu_ortho_rank import COEF, EPS, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,layout,grad_dtype", FFN_VARIANTS)
@pytest.mark.parametrize("T,H,I", FFN_SHAPES)
def test_feed_forward_block(T, H, I, act, layout, grad_dtype):
    run(inputs(T, H, I, seed=T, xscale=3.0 if act == "clamped" else 1.0), act, layout, grad_dtype)


def stack(E, M, N, seed):
    """Gradients of a few strong directions over noise."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = min(8, M, N)
    low = torch.randn(E, M, r, generator=g, device="cuda") @ torch.randn(E, r, N, generator=g, device="cuda")
    return (low + torch.randn(E, M, N, generator=g, device="cuda")) * 1e-4


@pytest.mark.parametrize("E,M,N", STACKS)
def test_orthogonalisation_and_step(E, M, N):
    """Some matrices of each stack, the first and the last among them."""
    u = stack(E, M, N, seed=E)
    some = sorted({0, E // 3, E - 1}) if E * M * N < 1 << 25 else [0, E - 1]
    narrow = min(M, N) < 64   # roundings do not average out
    wide = torch.full((E, M, N), float("nan"), device="cuda")
    moe.orthogonalize(u, dtype="fp32", out=wide)
    half = torch.full((E, M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.orthogonalize(u, out=half)
    assert torch.isfinite(wide).all() and torch.equal(wide.bfloat16(), half)
    compare(wide[some], u[some], torch.float32, cap=2.0 ** -7 if narrow else 2.0 ** -8, average=not narrow)
    # a step whose update is u itself: w - X within fp32 sums, and within a rounding of w's type, of the above
    m = torch.zeros_like(u)
    for w_type in (torch.float32, torch.bfloat16):
        w = torch.randn(E, M, N, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(w_type)
        got, mom, _ = moe.muon_step(w, u, m, lr=1.0, momentum=0.0, nesterov=False, out=(torch.empty_like(w), torch.empty_like(m)))
        assert torch.equal(mom, u)
        want = w.double() - wide.double()
        assert ((got.double() - want).abs() <= half_step(w_type) * want.abs() + 2.0 ** -23 * (w.double().abs() + wide.double().abs())).all()


def test_singular_values_of_a_large_matrix():
    """What the operator is for, on the largest tiles."""
    u = stack(16, 520, 1040, seed=3)
    o, _ = moe.orthogonalize(u, dtype="fp32")
    x = newton_schulz(u[:2], COEF, 5, EPS)
    s, t = torch.linalg.svdvals(o[:2].double().cpu()), torch.linalg.svdvals(x.cpu())
    assert ((s - t).abs() <= 2.0 ** -8 * t.norm(dim=-1, keepdim=True)).all()
