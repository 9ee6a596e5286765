"""A whole block with its operators called one after the other, as a program calls them: norm, routed experts beside a
shared expert, residual step with the next norm; its backward pass; an optimiser step on the experts' gradients; and a
token decoded on the serving forms.  In fp32 against the same block in float64 by automatic differentiation.

Tolerance: each step is an fp32 computation of sums of at most a few hundred terms of one size, so its relative error in
the 2-norm is below sqrt(n) 2^-24 < 2^-19, and the hardware's exp and reciprocal add up to 2^-17 in phi; eight steps in a
row, each amplifying what came in by at most about 4, stay below 2^-10."""
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
from tests._block import newton_schulz

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -10
T, H, I, E, K = 40, 72, 40, 5, 2
SCALE, EPS = 0.7, 1e-5


def make(T=T, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).cuda()  # noqa: E731
    return dict(x=r(T, H), w_in=1 + r(H, std=0.2), wr=r(E, H, std=H ** -0.5), gu=r(E, 2 * I, H, std=H ** -0.5), dn=r(E, H, I, std=I ** -0.5),
                sgu=r(2 * I, H, std=H ** -0.5), sdn=r(H, I, std=I ** -0.5), wg=r(H, std=H ** -0.5), w_post=1 + r(H, std=0.2),
                w_next=1 + r(H, std=0.2), d_new=r(T, H), d_y=r(T, H))


def rms(v, w):
    return w * v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)


def expert(y, gu, dn):
    g, u = (y @ gu.T).chunk(2, -1)
    return (g * torch.sigmoid(g) * u) @ dn.T


def reference(p, ids):
    """(x_new, y_next) in float64; the choice of experts is given."""
    y = rms(p["x"], p["w_in"])
    w = torch.softmax(torch.gather(y @ p["wr"].T, 1, ids), 1)
    every = torch.stack([expert(y, p["gu"][e], p["dn"][e]) for e in range(E)], 1)   # [T, E, H]
    routed = (torch.gather(every, 1, ids[..., None].expand(-1, -1, H)) * w[..., None]).sum(1)
    h = routed + torch.sigmoid(y @ p["wg"])[:, None] * expert(y, p["sgu"], p["sdn"])
    new = p["x"] + SCALE * rms(h, p["w_post"])
    return new, rms(new, p["w_next"])


def close(got, want, name):
    d, n = (got.double() - want).norm().item(), want.norm().item()
    assert d <= TOL * n, f"{name}: {d / n:.3e}"


def forward(p, save=True):
    y = moe.norm_fwd(p["x"], p["w_in"], eps=EPS)
    logits, gate = y @ p["wr"].T, y @ p["wg"]
    routed, ids, w, zr, _ = moe.fwd_logits(y, logits, K, p["gu"], p["dn"], save=save)
    h, zs, _ = moe.ffn_fwd(y, p["sgu"], p["sdn"], gate=gate, add=routed, save=save)
    new, nxt = moe.residual_fwd(p["x"], h, w_post=p["w_post"], scale=SCALE, w_next=p["w_next"], eps=EPS)
    return dict(y=y, gate=gate, ids=ids, w=w, zr=zr, zs=zs, h=h, new=new, next=nxt)


def test_forward_backward_and_step():
    p = make()
    f = forward(p)
    leaves = {k: v.double().requires_grad_(k not in ("d_new", "d_y")) for k, v in p.items()}
    new, nxt = reference(leaves, f["ids"].long())
    close(f["new"], new.detach(), "x_new")
    close(f["next"], nxt.detach(), "y")
    names = [k for k in leaves if k not in ("d_new", "d_y")]
    want = dict(zip(names, torch.autograd.grad((new, nxt), [leaves[k] for k in names], (leaves["d_new"], leaves["d_y"]))))

    r = moe.residual_bwd(f["new"], f["h"], p["d_new"], p["d_y"], w_post=p["w_post"], scale=SCALE, w_next=p["w_next"], eps=EPS)
    dys, dgate, dsgu, dsdn, _ = moe.ffn_bwd(f["y"], p["sgu"], p["sdn"], r.d_h, saved=f["zs"], gate=f["gate"])
    dyr, dw, dgu, ddn, _ = moe.bwd(f["y"], f["ids"], f["w"], p["gu"], p["dn"], r.d_h, saved=f["zr"])
    dlog = moe.router_bwd(f["ids"], f["w"], dw, E)
    dy = dys + dyr + dlog @ p["wr"] + dgate[:, None] * p["wg"]
    dx, dwin, _ = moe.norm_bwd(p["x"], p["w_in"], dy, d_add=r.d_x, eps=EPS)
    got = dict(x=dx, w_in=dwin, wr=dlog.T @ f["y"], gu=dgu, dn=ddn, sgu=dsgu, sdn=dsdn, wg=dgate @ f["y"], w_post=r.d_w_post,
               w_next=r.d_w_next)
    for k in names:
        close(got[k], want[k], "gradient of " + k)

    # a step of the stacked expert weights and of the shared ones (a stack of one), each towards its orthogonalised gradient
    for w, grad in ((p["gu"], dgu), (p["dn"], ddn), (p["sgu"], dsgu)):
        m = torch.zeros_like(w)
        w1, m1, _ = moe.muon_step(w, grad, m, lr=0.1, momentum=0.9, nesterov=False, out=(torch.empty_like(w), torch.empty_like(m)))
        assert torch.equal(m1, grad)
        o = newton_schulz(grad, moe.NEWTON_SCHULZ, 5, 1e-7)
        off = newton_schulz(grad, moe.NEWTON_SCHULZ, 5, 1e-7, half=True) - o
        step = (w.double() - w1.double()) / 0.1
        assert (step - o).norm() <= 2 * off.norm() + 2.0 ** -19 * (o.norm() + w.double().norm() / 0.1)


@pytest.mark.parametrize("T", [1, 3, 16])
def test_decoding(T):
    """The serving forms of the same block give what the training forms give."""
    p = make(T, seed=T)
    f = forward(p, save=False)
    y = moe.norm_fwd(p["x"], p["w_in"], eps=EPS)
    routed, ids, _, _ = moe.fwd_few_logits(y, y @ p["wr"].T, K, p["gu"], p["dn"])
    h, _, _ = moe.ffn_fwd(y, p["sgu"], p["sdn"], gate=y @ p["wg"], add=routed, out=routed)
    new, nxt = moe.residual_fwd(p["x"], h, w_post=p["w_post"], scale=SCALE, w_next=p["w_next"], eps=EPS, x_new=p["x"])
    assert torch.equal(ids, f["ids"])
    close(new, f["new"].double(), "x_new")
    close(nxt, f["next"].double(), "y")
    leaves = {k: v.double() for k, v in make(T, seed=T).items()}
    want, _ = reference(leaves, ids.long())
    close(new, want, "x_new against float64")


def test_block_captured_and_replayed():
    """The block's forward pass in one graph: every replay equals the eager calls on the same input."""
    p = make(seed=3)
    for _ in range(2):
        forward(p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = forward(p)
    for k in range(3):
        p["x"].copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(20 + k)))
        e = forward(p)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(f["new"], e["new"]) and torch.equal(f["next"], e["next"])
