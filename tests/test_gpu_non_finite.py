"""Weights that are not finite, through every forward and the backward: what the layer computes is NaN wherever the
formula's is, also where a clamp stands between (min and clamp of a NaN are NaN).

The expected places come from the formula in 64 bits (numpy's minimum and clip keep a NaN).  A NaN in one gate or up row
of an expert makes one activation column of all its slots NaN, and with it every output of its tokens; no other token
changes by a bit."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
import oracle
from tests._gpu import device_inputs, host, small_inputs

pytestmark = pytest.mark.gpu

E = 4
BAD = 2   # the expert that holds the value


def routed(T, E=E):
    """Experts by turns; a single token goes to the expert under test."""
    return (np.arange(T) % E if T > 1 else np.array([BAD])).astype(np.int32).reshape(T, 1)


def row_of(part, layout, I, j):
    return (2 * j + (part == "up")) if layout == "interleaved" else j + (I if part == "up" else 0)


def check(run, ids, put):
    """run(): the layer's output; put(): sets a weight of the expert to NaN."""
    want = host(run())
    assert np.all(np.isfinite(want))
    put()
    got = host(run())
    hit = np.any(ids == BAD, axis=1)
    assert np.all(np.isnan(got[hit]))
    assert np.array_equal(got[~hit], want[~hit])


@pytest.mark.parametrize("part", ["gate", "up"])
@pytest.mark.parametrize("layout", ["concat", "interleaved"])
@pytest.mark.parametrize("T,E", [(1, 4), (6, 4), (80, 4), (140, 9), (400, 4)])
def test_nan_block_of_a_4_bit_row(T, E, layout, part):
    """Scale byte 255 in one block of one gate or up row: one token, the few-token kernels with one column tile and with
    two, and the grouped products on tiles of 32 and of 64 positions."""
    H, I = 160, 96
    ids = routed(T, E)
    inp = small_inputs(T, H, I, E, 1, "bf16", "clamped", layout, seed=T, ids=ids)
    gu, dn = (moe.mx_quantize(torch.from_numpy(v).cuda()) for v in (inp.w_gate_up, inp.w_down))
    x, w = torch.from_numpy(inp.hidden).cuda().bfloat16(), torch.from_numpy(inp.topk_weights).cuda()
    i = torch.from_numpy(ids).cuda()

    def put():
        gu[1][BAD, row_of(part, layout, I, 37), 3] = 255

    check(lambda: moe.mx_fwd(x, i, w, gu, dn, act="clamped", layout=layout)[0], ids, put)


@pytest.mark.parametrize("part", ["gate", "up"])
@pytest.mark.parametrize("layout", ["concat", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 6, 80])
def test_nan_weight_for_a_few_tokens(T, dtype, layout, part):
    ids = routed(T)
    inp = small_inputs(T, 136, 72, E, 1, dtype, "clamped", layout, seed=T, ids=ids)
    d = device_inputs(inp)

    def put():
        d["w_gate_up"][BAD, row_of(part, layout, 72, 37), 90] = float("nan")

    check(lambda: moe.fwd_few(d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"], act="clamped",
                              layout=layout)[0], ids, put)


@pytest.mark.parametrize("act", ["clamped", "swiglu"])
def test_infinite_activation_on_a_zero_up_weight(act):
    """inf * 0 in the up sum alone: the gate's sum is +inf, which a clamp makes finite, the up's is NaN."""
    H, I, T = 64, 32, 5
    inp = small_inputs(T, H, I, E, 1, "fp32", act, "concat", seed=3, ids=routed(T))
    inp.w_gate_up[:, :I, 7] = 0.5
    inp.w_gate_up[:, I:, 7] = 0.0
    inp.hidden[1, 7] = np.inf
    d = device_inputs(inp)
    q = [moe.mx_quantize(d[n]) for n in ("w_gate_up", "w_down")]
    r = [d["topk_ids"], d["topk_weights"]]
    outs = [moe.fwd_few(d["hidden"], *r, d["w_gate_up"], d["w_down"], act=act)[0],
            moe.fwd(d["hidden"], *r, d["w_gate_up"], d["w_down"], act=act)[0],
            moe.mx_fwd(d["hidden"].bfloat16(), *r, *q, act=act)[0]]
    for out in outs:
        out = host(out)
        assert np.all(np.isnan(out[1])) and np.all(np.isfinite(np.delete(out, 1, axis=0)))


# fp32, register-staged and LDS-DMA tiles of 128 rows and the 256-row ones (experts of 600 slots)
SIZES = [("fp32", 40, 72, 40), ("bf16", 40, 136, 72), ("bf16", 200, 128, 64), ("bf16", 2400, 288, 160), ("bf16", 2400, 128, 64)]


@pytest.mark.parametrize("dtype,T,H,I", SIZES)
@pytest.mark.parametrize("part", ["gate", "up"])
@pytest.mark.parametrize("layout", ["concat", "interleaved"])
def test_nan_weight_in_the_forward(dtype, T, H, I, layout, part):
    ids = routed(T)
    inp = small_inputs(T, H, I, E, 1, dtype, "clamped", layout, seed=T + H, ids=ids)
    d = device_inputs(inp)

    def put():
        d["w_gate_up"][BAD, row_of(part, layout, I, 37), 60] = float("nan")

    check(lambda: moe.fwd(d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"], act="clamped",
                          layout=layout)[0], ids, put)


@pytest.mark.parametrize("dtype,T,H,I", SIZES)
@pytest.mark.parametrize("save", [True, False])
@pytest.mark.parametrize("layout", ["concat", "interleaved"])
def test_nan_up_weight_in_the_backward(dtype, T, H, I, layout, save):
    """Every gradient is NaN where the formula's is and nowhere else.  (A NaN up value is outside its clamp's interval, so
    the clamp passes no gradient to that row, as in the formula; the gate's row, the down column, the tokens and
    their routing weights are NaN.)"""
    inp = small_inputs(T, H, I, E, 1, dtype, "clamped", layout, seed=T + H, ids=routed(T))
    inp.w_gate_up[BAD, row_of("up", layout, I, 37), 60] = np.nan
    d = device_inputs(inp)
    r = (d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"])
    kw = dict(act="clamped", layout=layout)
    saved = moe.fwd(*r, save=True, **kw)[1] if save else None
    got = moe.bwd(*r, d["d_out"], saved=saved, **kw)[:4]
    with np.errstate(invalid="ignore"):
        ref = oracle.backward(inp.hidden, inp.topk_ids, inp.topk_weights, inp.dout,
                              oracle.expert_accessor(inp.w_gate_up, inp.w_down), E, "clamped", layout)
    for name, g, want in zip(("d_hidden", "d_topk_weights", "d_w_gate_up", "d_w_down"), got, ref):
        assert np.array_equal(np.isnan(host(g)), np.isnan(want)), name
