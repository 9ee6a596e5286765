"""Orthogonalisation of updates of any rank and spread of singular values, as weight gradients are: that of an expert
with n slots has rank n at most.  What rounding puts outside of an update's range grows with every step, by 485 in five.

Against 64 bits, within
* twice what the kernels' roundings do to the iteration in 64 bits (fp32 sums in another order and the roundings of values
  near a tie fall differently), and for fp32 sums and products, off by a few half steps of 2^-24, 2^-21 times what grows
  outside of the range, a^steps (2^-12 in five steps);
* 2^-8 whatever the emulation says: a rounding to 11 bits is off by 2^-12 in the mean, of the terms |b| s^2 + 2 |c| s^4
  (P's) and |b s^2 + c s^4| (Q's, X's high half) at singular values s of about one, 11.6 in all, over the result's 0.7 to
  1.2, and two steps' worth of it remains: 2^-12 times 11.6 sqrt(2) = 2^-8."""
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
from tests._block import half_step, newton_schulz

pytestmark = pytest.mark.gpu
COEF, EPS = moe.NEWTON_SCHULZ, 1e-7


def held(t, scale):
    """As fp16 times scale holds it."""
    return (t * scale).half().double() / scale


def rounded(u, coef, steps, eps):
    """The iteration with the kernels' roundings: X as a pair of fp16 values whose high half the products take, P and Q in
    fp16 with their diagonals kept; a X, in the last two steps the whole diagonal of Q, on the pair."""
    a, b, c = coef
    x = u.double() / (u.double().square().sum((-2, -1), keepdim=True).sqrt() + eps)
    flip = x.shape[-2] > x.shape[-1]
    if flip:
        x = x.mT.contiguous()
    for i in range(steps):
        high = held(x, 64.0)
        x = high + held(x - high, 64.0 * 2048)
        p = high @ high.mT.contiguous()
        stored = held(p, 4096.0)
        d = stored.diagonal(dim1=-2, dim2=-1)
        q = b * stored + c * (stored @ stored)
        whole = q.diagonal(dim1=-2, dim2=-1) + (b + 2 * c * d) * (p.diagonal(dim1=-2, dim2=-1) - d)
        kept = whole if i + 2 < steps else torch.zeros_like(whole)
        q = held(q - torch.diag_embed(q.diagonal(dim1=-2, dim2=-1) - kept), 4096.0)
        x = (a + whole - q.diagonal(dim1=-2, dim2=-1))[..., None] * x + q @ high
    return x.mT.contiguous() if flip else x


def update(M, N, kind, dtype, seed=0, E=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    S = min(M, N)
    if isinstance(kind, int):
        u = rand(E, M, kind) @ rand(E, kind, N)
    elif kind == "full":
        u = rand(E, M, N)
    elif kind == "one strong":   # one direction 1000 times the others
        u = rand(E, M, N) + 1000 * rand(E, M, 1) @ rand(E, 1, N)
    elif kind == "geometric":    # singular values from 1 to 1e-6
        q, _ = torch.linalg.qr(rand(E, M, S).cpu())
        r, _ = torch.linalg.qr(rand(E, N, S).cpu())
        u = ((q * torch.logspace(0, -6, S, dtype=torch.float64)) @ r.mT).cuda()
    elif kind == "rows":         # a gradient in a few rows only
        u = torch.zeros(E, M, N, dtype=torch.float64, device="cuda")
        u[:, 1:4] = rand(E, 3, N)
    else:                        # a few slots, two of them much alike
        u = rand(E, M, 4) @ rand(E, 4, N)
        u[:, :, N // 2:] = 0
    return (u * 1e-4).to(dtype)


def compare(got, u, dtype, steps=5, coef=COEF, cap=2.0 ** -8, average=True):
    exact = newton_schulz(u, coef, steps, EPS)
    off = torch.linalg.vector_norm(rounded(u, coef, steps, EPS) - exact, dim=(-2, -1))
    n = torch.linalg.vector_norm(exact, dim=(-2, -1))
    d = torch.linalg.vector_norm(got.double() - exact, dim=(-2, -1))
    rest = half_step(dtype) if dtype == torch.bfloat16 else 0.0
    assert not average or (d <= 2 * off + (2.0 ** -21 * coef[0] ** steps + rest) * n).all(), f"{(d / n).max().item():.2e}, emulated {(off / n).max().item():.2e}"
    assert cap is None or (d <= (cap + rest) * n).all(), f"{(d / n).max().item():.2e}"


KINDS = [1, 2, 8, 64, "half", "full", "one strong", "geometric", "rows", "slots"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("g_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N", [(512, 512), (104, 1000), (1000, 104), (328, 712)])
def test_any_rank(M, N, kind, g_type):
    u = update(M, N, min(M, N) // 2 if kind == "half" else kind, g_type, seed=M + N)
    o, _ = moe.orthogonalize(u, dtype="fp32")
    compare(o, u, torch.float32)
    o, _ = moe.orthogonalize(u)
    compare(o, u, torch.bfloat16)


@pytest.mark.parametrize("M,N", [(8, 264), (264, 8), (24, 24), (56, 200), (200, 48), (64, 64)])
@pytest.mark.parametrize("kind", [1, 2, "full", "slots"])
def test_few_rows(M, N, kind):
    """Matrices of few elements, whose roundings do not average out: P and Q of 8 rows have 56 elements off their diagonals,
    of which two can be most of the error, and an fp32 sum 2^-24 beside a tie rounds the other way, so the emulation says
    nothing about a single matrix.  A rounding to 11 bits is off by 2^-11 at most, twice the mean above: 2^-7."""
    u = update(M, N, kind, torch.float32, seed=M + N, E=7)
    o, _ = moe.orthogonalize(u, dtype="fp32")
    compare(o, u, torch.float32, cap=2.0 ** -7, average=False)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 7])
@pytest.mark.parametrize("M,N", [(136, 264), (264, 136)])
def test_numbers_of_steps(steps, M, N):
    u = update(M, N, 3, torch.float32, seed=steps)
    for coef in (COEF, (2.0, -1.5, 0.5)):
        o, _ = moe.orthogonalize(u, steps=steps, coef=coef, dtype="fp32")
        compare(o, u, torch.float32, steps, coef, cap=None)


@pytest.mark.parametrize("M,N", [(2880, 1448), (1448, 2880)])
@pytest.mark.parametrize("kind", [4, 128])
def test_an_experts_size(M, N, kind):
    u = update(M, N, kind, torch.float32, seed=kind, E=1)
    o, _ = moe.orthogonalize(u, dtype="fp32")
    compare(o, u, torch.float32)


@pytest.mark.parametrize("w_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N", [(512, 328), (104, 1000)])
def test_step_of_an_expert_with_few_slots(M, N, w_type):
    u = update(M, N, 5, torch.float32)
    w = torch.randn(u.shape, generator=torch.Generator().manual_seed(1)).to(w_type).cuda() * 0.02
    m = torch.zeros_like(u)
    w1, m1, _ = moe.muon_step(w, u, m, lr=1.0, momentum=0.5, nesterov=True, out=(torch.empty_like(w), torch.empty_like(m)))
    assert torch.equal(m1, u)
    x = newton_schulz(1.5 * u.double(), COEF, 5, EPS)
    want = w.double() - x
    n = torch.linalg.vector_norm(x, dim=(-2, -1))
    d = torch.linalg.vector_norm(w1.double() - want, dim=(-2, -1))
    assert (d <= 2.0 ** -8 * n + half_step(w_type) * torch.linalg.vector_norm(want, dim=(-2, -1))).all(), (d / n).tolist()
