"""The block of tests/test_gpu_block.py within a tolerance that a lost gradient term would not pass.

Derived per operator, in the 2-norm: phi and its slopes are off by 2^-17 of a value (hardware exp and reciprocal), dZ by
twice that; fp32 sums of up to 72 terms of one size by less than 2^-20; products pass relative errors on unchanged, the
norms' gradients (a value less its projection, over rms) by at most twice, the choice's softmax (a difference of two
weighted terms) by at most four times: 4 * 2 * 2^-16 = 2^-13 for what passes all of them."""
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
from tests.test_gpu_block import EPS, SCALE, E, forward, make, reference

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -13


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("seed", [0, 1])
def test_every_term_counts(seed):
    p = make(seed=seed)
    f = forward(p)
    leaves = {k: v.double().requires_grad_(k not in ("d_new", "d_y")) for k, v in p.items()}
    new, nxt = reference(leaves, f["ids"].long())
    assert off(f["new"], new.detach()) <= TOL and off(f["next"], nxt.detach()) <= TOL
    names = [k for k in leaves if k not in ("d_new", "d_y")]
    want = dict(zip(names, torch.autograd.grad((new, nxt), [leaves[k] for k in names], (leaves["d_new"], leaves["d_y"]))))
    r = moe.residual_bwd(f["new"], f["h"], p["d_new"], p["d_y"], w_post=p["w_post"], scale=SCALE, w_next=p["w_next"], eps=EPS)
    dys, dgate, dsgu, dsdn, _ = moe.ffn_bwd(f["y"], p["sgu"], p["sdn"], r.d_h, saved=f["zs"], gate=f["gate"])
    dyr, dw, dgu, ddn, _ = moe.bwd(f["y"], f["ids"], f["w"], p["gu"], p["dn"], r.d_h, saved=f["zr"])
    dlog = moe.router_bwd(f["ids"], f["w"], dw, E)
    terms = dict(shared=dys, routed=dyr, router=dlog @ p["wr"], gate=dgate[:, None] * p["wg"])

    def into_x(terms, d_add):
        return moe.norm_bwd(p["x"], p["w_in"], sum(terms.values()), d_add=d_add, eps=EPS)[:2]
    dx, dwin = into_x(terms, r.d_x)
    got = dict(x=dx, w_in=dwin, wr=dlog.T @ f["y"], gu=dgu, dn=ddn, sgu=dsgu, sdn=dsdn, wg=dgate @ f["y"], w_post=r.d_w_post,
               w_next=r.d_w_next)
    for k in names:
        assert off(got[k], want[k]) <= TOL, (k, off(got[k], want[k]))
    # a gradient that lacks one of its terms is far outside
    for lost in terms:
        without = into_x({k: v for k, v in terms.items() if k != lost}, r.d_x)
        assert off(without[0], want["x"]) > 32 * TOL and off(without[1], want["w_in"]) > 32 * TOL, lost
    assert off(into_x(terms, None)[0], want["x"]) > 32 * TOL
