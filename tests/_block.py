"""64-bit references, with error bounds, of the operators around the routed
experts (torch in float64, on the inputs' device).

Every bound is first order and worst case; `u` is half a step of the stored
type (2^-8 bf16, 2^-24 fp32), E = 2^-24 one fp32 rounding.  An fp32 sum of n
terms is off by at most n E times the sum of the terms' sizes in any order.
The factor SECOND covers products of two such errors.
"""
import torch

E = 2.0 ** -24
SECOND = 1.02


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, ref, bound, name=""):
    """Elementwise within the bound; nothing non-finite where the reference is finite."""
    got = got.double()
    assert got.shape == ref.shape, name
    assert torch.isfinite(got).all(), f"{name}: non-finite values"
    over = (got - ref).abs() - bound
    if over.numel():
        assert over.max().item() <= 0, f"{name}: {over.max().item():.3e} past the bound at {over.argmax().item()} of {tuple(ref.shape)}"


def check_norm(got, ref, tol, name=""):
    n = ref.norm().item()
    d = (got.double() - ref).norm().item()
    assert d <= tol * n, f"{name}: {d / n if n else d:.3e} of {tol:.3e} in the 2-norm"


# ------------------------------------------------------------------ feed-forward block
def _halves(z, layout):
    return (z[..., 0::2], z[..., 1::2]) if layout == "interleaved" else z.chunk(2, dim=-1)


def _whole(g, u, layout):
    return torch.stack((g, u), -1).flatten(-2) if layout == "interleaved" else torch.cat((g, u), -1)


class Ffn:
    """out and gradients of the block in 64 bits, and what an implementation may be off by: fp32 sums, phi(..) and dZ
    rounded to the activations' type as operands, results to theirs.

    phi = f(g) v(u): f(g) = g sigmoid(al g), v = u (swiglu, al = 1) or f(min(g, L)), v = clamp(u) + 1.  |f'| <= 1.1,
    |f''| <= al / 2.  Hardware exp2 and reciprocal: 2^-17 of a value, arguments up to 2^6.  A gate or up value within
    its own error of a clamp may fall on either side, which counts as the whole slope there."""

    def __init__(self, x, gu, dn, act, layout, gate=None, add=None, limit=7.0, alpha=1.702):
        self.dt = x.dtype
        self.u = half_step(x.dtype)
        self.x, self.gu, self.dn, self.layout = x.double(), gu.double(), dn.double(), layout
        T, H = x.shape
        I = dn.shape[1]
        self.H, self.I, self.T = H, I, T
        g, u = _halves(self.x @ self.gu.T, layout)
        self.eg, self.eu = _halves(H * E * (self.x.abs() @ self.gu.abs().T), layout)
        al = 1.0 if act == "swiglu" else alpha
        gc = g if act == "swiglu" else g.clamp(max=limit)
        s = torch.sigmoid(al * gc)
        f, f1 = gc * s, s + al * gc * s * (1 - s)
        if act == "swiglu":
            v, v1 = u, torch.ones_like(u)
            self.jump_g = self.jump_u = torch.zeros_like(u)
        else:
            v, v1 = u.clamp(-limit, limit) + 1, (u.abs() <= limit).double()
            self.jump_g = ((g - limit).abs() <= self.eg).double() * f1.abs()
            self.jump_u = ((u.abs() - limit).abs() <= self.eu).double()
            f1 = f1 * (g <= limit)
        self.f, self.v, self.f1, self.v1, self.al = f, v, f1, v1, al
        self.a = f * v
        self.ea = SECOND * (1.1 * v.abs() * self.eg + f.abs() * self.eu + 2.0 ** -17 * self.a.abs())
        self.s = torch.sigmoid(gate.double()) if gate is not None else torch.ones(T, dtype=torch.float64, device=x.device)
        self.es = 2.0 ** -21 * self.s if gate is not None else torch.zeros_like(self.s)
        y = self.a @ self.dn.T
        ey = (self.ea + self.u * self.a.abs()) @ self.dn.abs().T + (I + 4) * E * (self.a.abs() @ self.dn.abs().T)
        ad = add.double() if add is not None else torch.zeros_like(y)
        self.out = ad + self.s[:, None] * y
        err = self.s[:, None] * ey + self.es[:, None] * y.abs() + 2 * E * (ad.abs() + y.abs())
        self.out_bound = SECOND * (err + self.u * self.out.abs() + self.u * err)

    def backward(self, dout, grad_dtype):
        d = dout.double()
        s = self.s[:, None]
        ug = half_step(grad_dtype)
        r = d @ self.dn
        er = self.H * E * (d.abs() @ self.dn.abs())
        da = s * r
        eda = s * er + self.es[:, None] * r.abs()
        dg, du = da * self.f1 * self.v, da * self.f * self.v1
        edg = (eda * self.f1.abs() * self.v.abs() + da.abs() * (self.al / 2 * self.eg * self.v.abs() + 1.1 * self.eu
               + self.jump_g * self.v.abs()) + 2.0 ** -16 * dg.abs())
        edu = eda * self.f.abs() + da.abs() * (1.1 * self.eg + self.jump_u * self.f.abs()) + 2.0 ** -16 * du.abs()
        dz = _whole(dg, du, self.layout)
        edz = SECOND * _whole(edg, edu, self.layout) + self.u * dz.abs()
        sa = s * self.a
        esa = SECOND * (s * self.ea + self.es[:, None] * self.a.abs()) + self.u * sa.abs()
        got = {}

        def put(name, ref, err, u):
            got[name] = (ref, SECOND * (err + u * ref.abs() + u * err))
        put("d_x", dz @ self.gu, edz @ self.gu.abs() + 2 * self.I * E * (dz.abs() @ self.gu.abs()), self.u)
        put("d_gu", dz.T @ self.x, edz.T @ self.x.abs() + (self.T + 4) * E * (dz.abs().T @ self.x.abs()), ug)
        put("d_dn", d.T @ sa, d.abs().T @ esa + (self.T + 4) * E * (d.abs().T @ sa.abs()), ug)
        ra = r * self.a
        p = self.s * (1 - self.s)
        # s (1 - s): the subtraction is exact to one rounding of s's error
        put("d_gate", p * ra.sum(1), p * (er * self.a.abs() + r.abs() * self.ea + (self.I + 8) * E * ra.abs()).sum(1)
            + (2 * self.es + 4 * E * self.s) * ra.sum(1).abs(), E)
        return got


# ------------------------------------------------------------------ norms
# A statistic is a sum of products by threads (16 terms each), wave steps and waves: below 64 roundings in a row, and
# the square root, quotient and products after it below 16.
STAT = 80 * E


class Norm:
    """n(v, w) = w v / rms(v) and its gradient, with bounds."""

    def __init__(self, v, w, eps):
        self.v, self.w = v.double(), w.double()
        self.r = 1 / torch.sqrt((self.v ** 2).mean(-1, keepdim=True) + eps)
        self.hat = self.v * self.r
        self.n = self.w * self.hat
        self.en = STAT * self.n.abs()

    def grad(self, g, eg=0.0):
        """(gradient of v, its error, hat * g, its error) for a gradient g of n that is off by eg."""
        wg = self.w * g
        ewg = self.w.abs() * eg
        mean = (wg * self.hat).mean(-1, keepdim=True)
        emean = (ewg * self.hat.abs() + STAT * (wg * self.hat).abs()).mean(-1, keepdim=True)
        d = self.r * (wg - self.hat * mean)
        ed = self.r * (ewg + self.hat.abs() * emean + STAT * (wg.abs() + self.hat.abs() * mean.abs()))
        return d, ed, self.hat * g, self.hat.abs() * (eg + STAT * g.abs())


def column_sum(terms, err):
    """Sum over rows, and its bound: rows added up by up to 512 workgroups, their sums in 16 parts."""
    T = terms.shape[0]
    return terms.sum(0), SECOND * (err.sum(0) + (T / 512 + 64) * E * terms.abs().sum(0))


# ------------------------------------------------------------------ Newton-Schulz
def newton_schulz(u, coef, steps, eps, half=False):
    """The iteration in 64 bits; half: with X, X X^T and Q = a I + b X X^T + .. rounded to fp16 (scaled by 2^6 and 2^12)
    as the kernels hold them, for the size of the error that this brings."""
    a, b, c = coef
    x = u.double() / (u.double().square().sum((-2, -1), keepdim=True).sqrt() + eps)
    flip = x.shape[-2] > x.shape[-1]
    if flip:
        x = x.mT.contiguous()

    def hold(t, scale):
        return (t * scale).half().double() / scale if half else t
    x = hold(x, 64.0)
    for i in range(steps):
        p = hold(x @ x.mT.contiguous(), 4096.0)
        x = hold(a * torch.eye(p.shape[-1], dtype=p.dtype, device=p.device) + b * p + c * (p @ p), 4096.0) @ x
        if i + 1 < steps:
            x = hold(x, 64.0)
    return x.mT.contiguous() if flip else x
