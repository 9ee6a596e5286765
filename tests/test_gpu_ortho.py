"""Newton-Schulz orthogonalisation and the optimiser step against 64 bits.

The kernels hold X, X X^T and Q in fp16; how far that brings the result from the
exact iteration depends on the matrix, so the allowance is twice what the same
roundings do to the iteration in 64 bits (which leaves fp32 sums: 2^-24 sqrt(n)
against 2^-11), plus the result's own rounding."""
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
from tests._block import check, half_step, newton_schulz

pytestmark = pytest.mark.gpu
COEF, EPS = moe.NEWTON_SCHULZ, 1e-7
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def updates(E, M, N, dtype="bf16", seed=0, std=1e-4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = min(8, M, N)
    s = torch.exp(-0.3 * torch.arange(r, device="cuda"))
    low = (torch.randn(E, M, r, generator=g, device="cuda") * s) @ torch.randn(E, r, N, generator=g, device="cuda")
    return ((low + torch.randn(E, M, N, generator=g, device="cuda")) * std).to(TYPES[dtype])


def compare(got, u, dtype="bf16", steps=5, coef=COEF, eps=EPS, scale=1.0):
    """Each matrix, and each of its rows and columns, within the allowance of the 2-norm (three times for one row or
    column, whose roundings are fewer and vary more)."""
    exact = newton_schulz(u, coef, steps, eps)
    off = newton_schulz(u, coef, steps, eps, half=True) - exact
    got = got.double()
    assert torch.isfinite(got).all()
    rest = half_step(TYPES[dtype]) if dtype == "bf16" else 2.0 ** -20
    for dims, times in (((-2, -1), 1.0), ((-1,), 3.0), ((-2,), 3.0)):
        n = torch.linalg.vector_norm(exact, dim=dims)
        d = torch.linalg.vector_norm(got - exact, dim=dims)
        a = torch.linalg.vector_norm(off, dim=dims)
        if len(dims) == 1:   # a row's own error varies: at least the matrix's mean
            a = torch.maximum(a, a.square().mean(-1, keepdim=True).sqrt())
        over = d - times * (2 * a + rest * n)
        assert over.max().item() <= 0, f"{over.max().item():.3e} over, dims {dims}, allowance {times * (2 * a + rest * n).max().item():.3e}"


@pytest.mark.parametrize("E,M,N", [(1, 8, 8), (3, 8, 264), (3, 264, 8), (2, 64, 64), (5, 72, 200), (4, 200, 72), (24, 200, 712),
                                   (2, 712, 200), (1, 256, 256), (1, 264, 520), (1, 520, 264), (7, 192, 192), (2, 328, 320)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sizes(E, M, N, dtype):
    u = updates(E, M, N, dtype, seed=M + N)
    o, ws = moe.orthogonalize(u, out=torch.full((E, M, N), float("nan"), dtype=torch.bfloat16, device="cuda"))
    compare(o, u)
    f, _ = moe.orthogonalize(u, dtype="fp32", ws=ws.fill_(0xFF))
    compare(f, u, "fp32")
    assert torch.equal(f.bfloat16(), o)


# Stacks large enough for each kind of tile, with ragged sides
@pytest.mark.parametrize("E,M,N", [(4, 1032, 1544), (3, 1544, 1032), (16, 520, 1040), (2, 2056, 2056), (1, 2880, 1448), (1, 2888, 2880)])
def test_large_stacks(E, M, N):
    u = updates(E, M, N, seed=E)
    o, _ = moe.orthogonalize(u)
    compare(o, u)


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
@pytest.mark.parametrize("M,N", [(72, 136), (136, 72)])
def test_steps_and_coefficients(steps, M, N):
    u = updates(2, M, N, "fp32", seed=steps)
    for coef in (COEF, (1.875, -1.25, 0.375), (2.0, -1.5, 0.5)):
        o, _ = moe.orthogonalize(u, steps=steps, coef=coef, dtype="fp32")
        compare(o, u, "fp32", steps, coef)


def test_singular_values_near_one():
    """What the operator is for: singular values of the usual coefficients' result lie in [0.65, 1.25]."""
    o, _ = moe.orthogonalize(updates(2, 136, 264, "fp32"), dtype="fp32")
    s = torch.linalg.svdvals(o.double().cpu())
    assert s.min() > 0.65 and s.max() < 1.25


@pytest.mark.parametrize("std", [1e-30, 1e-20, 1e20, 1e30])
def test_gradients_of_any_size(std):
    """The norm is summed in 64 bits: squares past fp32's range do no harm."""
    u = updates(2, 72, 136, "fp32", std=std)
    o, _ = moe.orthogonalize(u, eps=0.0, dtype="fp32")
    compare(o, u, "fp32", eps=0.0)


def test_zero_and_non_finite_matrices():
    u = updates(4, 72, 136, seed=1)
    want, _ = moe.orthogonalize(u)
    u[1] = 0
    u[2, 3, 4] = float("nan")
    got, _ = moe.orthogonalize(u)
    assert not got[1].any() and torch.isnan(got[2]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])


@pytest.mark.parametrize("g_type", ["bf16", "fp32"])
@pytest.mark.parametrize("w_type", ["bf16", "fp32"])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("E,M,N", [(3, 72, 200), (2, 264, 136)])
def test_optimiser_step(g_type, w_type, nesterov, E, M, N):
    g, m = updates(E, M, N, g_type, seed=1), updates(E, M, N, "fp32", seed=2) * 4
    w = (torch.randn(E, M, N, generator=torch.Generator().manual_seed(3)) * 0.02).to(TYPES[w_type]).cuda()
    lr, mu, decay = 0.02, 0.95, 0.01
    kw = dict(lr=lr, momentum=mu, nesterov=nesterov, decay=decay)
    w1, m1, _ = moe.muon_step(w, g, m, out=(torch.empty_like(w), torch.empty_like(m)), **kw)
    f32 = lambda v: torch.tensor(v, dtype=torch.float32).double().item()  # noqa: E731
    m64 = f32(mu) * m.double() + g.double()
    check(m1, m64, 2.0 ** -23 * (m64.abs() + (f32(mu) * m).double().abs()), "m")
    u = g.double() + f32(mu) * m64 if nesterov else m64
    exact = newton_schulz(u, COEF, 5, EPS)
    off = newton_schulz(u, COEF, 5, EPS, half=True) - exact
    want = (1 - f32(decay)) * w.double() - f32(lr) * exact
    a = 2 * torch.linalg.vector_norm(off, dim=(-2, -1)) * lr
    a = a + (half_step(w.dtype) + 2.0 ** -22) * torch.linalg.vector_norm(want, dim=(-2, -1)) + 2.0 ** -20 * lr * torch.linalg.vector_norm(exact, dim=(-2, -1))
    assert (torch.linalg.vector_norm(w1.double() - want, dim=(-2, -1)) <= a).all()
    # in place
    moe.muon_step(w, g, m, **kw)
    assert torch.equal(w, w1) and torch.equal(m, m1)


def test_captured_and_replayed():
    u = updates(3, 200, 328, seed=5)
    w, m = torch.zeros(3, 200, 328, device="cuda"), torch.zeros(3, 200, 328, device="cuda")
    out = (torch.empty_like(w), torch.empty_like(m))
    _, _, ws = moe.muon_step(w, u, m, lr=0.1, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.muon_step(w, u, m, lr=0.1, out=out, ws=ws)
    for k in range(3):
        u.copy_(updates(3, 200, 328, seed=10 + k))
        want = moe.muon_step(w, u, m, lr=0.1, out=(torch.empty_like(w), torch.empty_like(m)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_empty_stack_and_leading_dimensions():
    o, _ = moe.orthogonalize(torch.empty(0, 8, 16, device="cuda"))
    assert o.shape == (0, 8, 16)
    u = updates(6, 40, 24)
    a, _ = moe.orthogonalize(u)
    b, _ = moe.orthogonalize(u.view(2, 3, 40, 24))
    c, _ = moe.orthogonalize(u[4])
    assert torch.equal(b.view(6, 40, 24), a) and torch.equal(c, a[4])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_eps_of_zero(dtype):
    """Zero matrices stay zero, and subnormal ones, whose norm's reciprocal is past fp32's range, are orthogonalised."""
    u = updates(5, 64, 136, dtype, std=1.0)
    u[0] *= 2.0 ** -130
    u[2] = 0
    u[3] *= 2.0 ** 100
    o, _ = moe.orthogonalize(u, eps=0.0)
    assert torch.count_nonzero(o[2]) == 0
    keep = [0, 1, 3, 4]
    compare(o[keep], u[keep], eps=0.0)


def held_off_the_diagonal(u, steps):
    """The iteration with the kernels' roundings except those of the diagonals of X X^T and Q."""
    a, b, c = COEF

    def hold(t, scale, keep_diagonal):
        r = (t * scale).half().double() / scale
        return r - torch.diag_embed(r.diagonal(dim1=-2, dim2=-1) - t.diagonal(dim1=-2, dim2=-1)) if keep_diagonal else r
    x = u.double() / u.double().square().sum((-2, -1), keepdim=True).sqrt()
    x = hold(x.mT.contiguous() if x.shape[-2] > x.shape[-1] else x, 64.0, False)
    for i in range(steps):
        p = hold(x @ x.mT.contiguous(), 4096.0, True)
        x = hold(a * torch.eye(p.shape[-1], dtype=p.dtype, device=p.device) + b * p + c * (p @ p), 4096.0, True) @ x
        if i + 1 < steps:
            x = hold(x, 64.0, False)
    return x.mT.contiguous() if u.shape[-2] > u.shape[-1] else x


# Long matrices, whose singular values lie close together and pass where the iteration is steep (|f'| up to 4 at 1.2), so
# that roundings of the diagonals of X X^T and Q would be most of the error: within twice what the others bring.
@pytest.mark.parametrize("M,N", [(2120, 104), (96, 5760), (104, 2120), (96, 1000), (600, 64)])
def test_diagonals_are_not_rounded(M, N):
    u = updates(2, M, N, seed=M)
    exact = newton_schulz(u, COEF, 5, 0.0)
    off = (held_off_the_diagonal(u, 5) - exact).norm().item()
    o, _ = moe.orthogonalize(u, dtype="fp32", eps=0.0)
    assert (o.double() - exact).norm().item() <= 2 * off + 2.0 ** -20 * exact.norm().item()
