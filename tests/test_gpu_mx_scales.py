"""The layer on 4-bit weights at both ends of the scale byte's range, on every kernel that expands codes."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
from tests._gpu import host
from tests._serve import check_layer, layer_bound, values_ref

pytestmark = pytest.mark.gpu

H, I = 160, 96
# one token, few-token kernels, grouped products on tiles of 32 and 64 positions
SIZES = [(1, 4), (6, 4), (80, 4), (140, 9), (400, 4)]


def weights(E, gu_scales, dn_scales, seed):
    g = torch.Generator().manual_seed(seed)
    pick = lambda of, shape: torch.tensor(of, dtype=torch.uint8)[torch.randint(0, len(of), shape, generator=g)]
    gu = [torch.randint(0, 256, (E, 2 * I, H // 2), dtype=torch.uint8, generator=g), pick(gu_scales, (E, 2 * I, H // 32))]
    dn = [torch.randint(0, 256, (E, H, I // 2), dtype=torch.uint8, generator=g), pick(dn_scales, (E, H, I // 32))]
    return gu, dn, g


def tokens(T, E, g, scale):
    ids = (torch.arange(T) % E).to(torch.int32).reshape(T, 1)
    return (torch.randn(T, H, generator=g) * scale).bfloat16(), ids, torch.ones(T, 1)


def run(x, ids, w, gu, dn):
    return moe.mx_fwd(x.cuda(), ids.cuda(), w.cuda(), [t.cuda() for t in gu], [t.cuda() for t in dn])[0]


def compare(x, ids, w, gu, dn):
    vg, vd = (values_ref(q[0].numpy(), q[1].numpy()) for q in (gu, dn))
    with np.errstate(over="ignore"):
        ref, bound = layer_bound(x.float().numpy(), ids.numpy(), w.numpy(), list(zip(vg, vd)), "swiglu", "concat", "bf16")
    check_layer(host(run(x, ids, w, gu, dn)), ref, bound)


@pytest.mark.parametrize("T,E", SIZES)
def test_lowest_scales(T, E):
    """Bytes 0, 1 and 2: weights of 2^-128 to 1.5 * 2^-123, subnormal ones among them, on values that bring the sums back
    into range.  gate_up: hidden states near 2^120.  down: activations near 2^117 (gate and up near 2^58; silu of such a
    gate is the gate or 0)."""
    gu, dn, g = weights(E, [0, 1, 2], range(116, 122), T)
    compare(*tokens(T, E, g, 2.0 ** 120), gu, dn)
    gu, dn, g = weights(E, range(116, 122), [0, 1, 2], T)
    compare(*tokens(T, E, g, 2.0 ** 60), gu, dn)


@pytest.mark.parametrize("T,E", SIZES)
def test_highest_scales(T, E):
    """Bytes 253 and 254 with codes whose values both types hold (below 2^128), on hidden states near 2^-124."""
    gu, dn, g = weights(E, [253, 254], range(116, 122), T)
    most = torch.where(gu[1] == 254, 3, 5).repeat_interleave(16, dim=-1)   # 1.5 and 3
    low, high = gu[0] & 15, gu[0] >> 4
    gu[0] = ((torch.minimum(low & 7, most) | (low & 8)) | ((torch.minimum(high & 7, most) | (high & 8)) << 4)).to(torch.uint8)
    compare(*tokens(T, E, g, 2.0 ** -124), gu, dn)


@pytest.mark.parametrize("T,E", SIZES)
@pytest.mark.parametrize("scale,code", [(253, 6), (254, 4), (254, 7)])
def test_values_past_the_range(T, E, scale, code):
    """A weight of 2^128 and more is infinite, as it is when dequantised: the layer is that of the dequantised weights."""
    gu, dn, g = weights(E, range(116, 122), range(116, 122), T)
    gu[1][1, 7, 2], gu[0][1, 7, 32:48] = scale, 0
    gu[0][1, 7, 40] = code             # one gate weight of expert 1, column 80, the only one of its block
    dn[1][2, 5, 1], dn[0][2, 5, 16:32] = scale, 0
    dn[0][2, 5, 20] = code             # one down weight of expert 2, column 40
    x, ids, w = tokens(T, E, g, 1.0)
    if T == 1:
        ids[:] = 1
    x[:, 80] = 0.5
    got = host(run(x, ids, w, gu, dn))
    deq = [moe.mx_dequantize(*[t.cuda() for t in q]) for q in (gu, dn)]
    want = host(moe.fwd(x.cuda(), ids.cuda(), w.cuda(), *deq)[0])
    assert not np.all(np.isfinite(want))
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
