"""The layer for a few tokens (fwd_few) against the layer in 64 bits."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
from tests._gpu import device_inputs, host, small_inputs
from tests._serve import check_layer, layer_bound

pytestmark = pytest.mark.gpu


def run_case(inp, **extra):
    """fwd_few on poisoned outputs and workspace, against the reference."""
    wl = inp.wl
    d = device_inputs(inp)
    desc = moe.make_desc(wl.T, wl.H, wl.I, wl.E, inp.topk_ids.shape[1], wl.dtype, wl.act, wl.layout)
    ws = torch.full((moe.few_workspace_size(desc),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(d["hidden"], float("nan"))
    kw = dict(act=wl.act, layout=wl.layout)
    got, _ = moe.fwd_few(d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"], ws=ws, out=out, **kw)
    assert got is out
    again, _ = moe.fwd_few(d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"], **kw)
    torch.cuda.synchronize()
    assert torch.equal(got, again)
    ref, bound = layer_bound(inp.hidden, inp.topk_ids, inp.topk_weights, list(zip(inp.w_gate_up, inp.w_down)), wl.act,
                             wl.layout, wl.dtype)
    check_layer(host(got), ref, bound, wl.name)
    return got, ws


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 33, 48, 100, 128])
def test_token_counts(dtype, T):
    run_case(small_inputs(T, 136, 72, 9, 2, dtype, "clamped", "interleaved", seed=T))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,I", [(8, 8), (16, 24), (32, 16), (40, 264), (264, 40), (1048, 712), (512, 1032)])
def test_sizes(dtype, H, I):
    run_case(small_inputs(5, H, I, 6, 3, dtype, "swiglu", "concat", seed=H + I))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", ["swiglu", "clamped"])
@pytest.mark.parametrize("layout", ["concat", "interleaved"])
def test_activation_and_layout(dtype, act, layout):
    # inputs large enough that both clamps act
    run_case(small_inputs(7, 96, 56, 5, 2, dtype, act, layout, seed=3, xscale=12.0))


@pytest.mark.parametrize("E,K", [(1, 1), (3, 3), (200, 1), (200, 8), (1024, 4), (64, 64)])
def test_expert_counts(E, K):
    run_case(small_inputs(4, 64, 40, E, K, "bf16", "swiglu", "interleaved", seed=E))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("K", [1, 2, 3, 5, 8, 16, 17, 64])
def test_one_token(K, dtype):
    """One token's own kernels: fewer, as many and more slots than waves, and bad ids among them."""
    run_case(small_inputs(1, 136, 72, 64, K, dtype, "clamped", "interleaved", seed=K))
    run_case(small_inputs(1, 72, 200, 64, K, dtype, "swiglu", "concat", seed=K))
    ids = np.resize(np.array([3, -1, 3, 64, 5], dtype=np.int32), (1, K))
    got, ws = run_case(small_inputs(1, 40, 24, 64, K, dtype, "swiglu", "concat", seed=K, ids=ids))
    assert moe.check_device_status(ws) == (moe.MOE_ERR_BAD_EXPERT_ID if K > 1 else moe.MOE_OK)


@pytest.mark.parametrize("E", [1, 2, 5, 63, 64, 129, 1024])
def test_one_token_from_logits(E):
    """The choice inside one token's kernel is the router's: ties, infinities, NaN."""
    K = min(E, 6)
    inp = small_inputs(1, 64, 40, E, K, "bf16", "swiglu", "concat", seed=E)
    d = device_inputs(inp)
    g = torch.Generator().manual_seed(E)
    rows = [torch.randn(1, E, generator=g), torch.randint(0, 3, (1, E), generator=g).float(), torch.zeros(1, E),
            torch.full((1, E), float("-inf"))]
    nan = torch.randn(1, E, generator=g)
    nan[0, ::2] = float("nan")
    rows += [nan, torch.full((1, E), float("nan"))]
    for lg in rows:
        lg = lg.cuda()
        out, ids, w, ws = moe.fwd_few_logits(d["hidden"], lg, K, d["w_gate_up"], d["w_down"])
        rids, rw, *_, rws = moe.router(lg, K)
        assert torch.equal(ids, rids)
        assert torch.equal(w.view(torch.int32), rw.view(torch.int32)) or torch.equal(torch.isnan(w), torch.isnan(rw))
        assert moe.check_device_status(ws) == moe.check_device_status(rws)
        if torch.all(torch.isfinite(w)):
            assert torch.equal(out, moe.fwd_few(d["hidden"], ids, w, d["w_gate_up"], d["w_down"])[0])


@pytest.mark.parametrize("T", [16, 17, 32, 33, 48, 64, 65, 96, 97, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_one_expert_takes_every_token(T, dtype):
    ids = np.full((T, 1), 2, dtype=np.int32)
    inp = small_inputs(T, 72, 136, 4, 1, dtype, "clamped", "concat", seed=T, ids=ids)
    run_case(inp)


@pytest.mark.parametrize("T", [32, 33, 128])
def test_large_layer_of_few_experts(T):
    run_case(small_inputs(T, 1456, 1456, 2, 2, "bf16", "clamped", "interleaved", seed=T))


@pytest.mark.parametrize("T", [125, 128])
def test_sides_of_the_rule_of_many_slots(T):
    """S H I just below and above 2e9: the latter runs the forward's kernels."""
    run_case(small_inputs(T, 2304, 2304, 3, 3, "bf16", "clamped", "concat", seed=T))


def test_repeated_ids_of_one_token():
    """Every slot of every token on one expert: 8 slots a token, 128 x 8 on the expert."""
    ids = np.full((128, 8), 1, dtype=np.int32)
    run_case(small_inputs(128, 40, 24, 8, 8, "bf16", "swiglu", "concat", seed=1, ids=ids))
    ids = np.tile(np.array([[3, 3, 0]], dtype=np.int32), (2, 1))
    run_case(small_inputs(2, 40, 24, 200, 3, "bf16", "swiglu", "concat", seed=2, ids=ids))


@pytest.mark.parametrize("E", [5, 100])
def test_bad_ids_are_dropped_and_reported(E):
    ids = np.array([[0, -1, 2], [E, E + 7, -(2 ** 31)], [2 ** 31 - 1, 4, 4], [1, 2, 3]], dtype=np.int32)
    inp = small_inputs(4, 48, 32, E, 3, "bf16", "swiglu", "concat", seed=4, ids=ids)
    got, ws = run_case(inp)
    assert moe.check_device_status(ws) == moe.MOE_ERR_BAD_EXPERT_ID
    assert torch.all(got[1] == 0)   # a token without a valid slot
    good = small_inputs(4, 48, 32, E, 3, "bf16", "swiglu", "concat", seed=4)
    assert moe.check_device_status(run_case(good)[1]) == moe.MOE_OK


def test_non_finite_values_stay_with_their_token():
    """A NaN token, an infinite routing weight and an unused expert of NaNs touch nothing else."""
    T, H, I, E, K = 20, 136, 72, 6, 2
    ids = np.stack((np.arange(T) % 5, (np.arange(T) + 1) % 5), axis=1).astype(np.int32)
    inp = small_inputs(T, H, I, E, K, "bf16", "swiglu", "concat", seed=5, ids=ids)
    inp.w_gate_up[5] = np.nan
    inp.w_down[5] = np.inf
    ref, bound = layer_bound(inp.hidden, ids, inp.topk_weights, list(zip(inp.w_gate_up, inp.w_down)), "swiglu", "concat", "bf16")
    inp.hidden[3] = np.nan
    inp.topk_weights[7, 1] = np.inf
    d = device_inputs(inp)
    out, _ = moe.fwd_few(d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"])
    out = host(out)
    assert np.all(np.isnan(out[3])) and not np.any(np.isfinite(out[7]))
    rest = [t for t in range(T) if t not in (3, 7)]
    check_layer(out[rest], ref[rest], bound[rest])


def test_no_tokens():
    inp = small_inputs(1, 64, 32, 4, 2, "bf16", "swiglu", "concat")
    d = device_inputs(inp)
    out, ws = moe.fwd_few(d["hidden"][:0], d["topk_ids"][:0], d["topk_weights"][:0], d["w_gate_up"], d["w_down"])
    assert tuple(out.shape) == (0, 64)
    assert moe.check_device_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("T,E,K", [(1, 128, 4), (3, 7, 7), (16, 256, 8), (128, 33, 2)])
def test_from_logits(T, E, K):
    """The logits form chooses what the router chooses and equals the form on those ids."""
    inp = small_inputs(T, 64, 40, E, K, "bf16", "clamped", "interleaved", seed=T)
    d = device_inputs(inp)
    lg = torch.randn(T, E, generator=torch.Generator().manual_seed(T)).cuda()
    if E >= 5:
        lg[:, 1] = lg[:, 4]   # ties
    kw = dict(act="clamped", layout="interleaved")
    out, ids, w, ws = moe.fwd_few_logits(d["hidden"], lg, K, d["w_gate_up"], d["w_down"], **kw)
    rids, rw = moe.router(lg, K)[:2]
    assert torch.equal(ids, rids) and torch.equal(w, rw)
    ref, _ = moe.fwd_few(d["hidden"], rids, rw, d["w_gate_up"], d["w_down"], **kw)
    assert torch.equal(out, ref)
    assert moe.check_device_status(ws) == moe.MOE_OK


def test_tokens_without_finite_logits():
    """A row of NaN logits has no choice: its ids are -1 and its output 0, the others are as without it."""
    inp = small_inputs(3, 64, 40, 8, 2, "bf16", "swiglu", "concat", seed=9)
    d = device_inputs(inp)
    lg = torch.randn(3, 8, generator=torch.Generator().manual_seed(1)).cuda()
    ref = moe.fwd_few_logits(d["hidden"], lg, 2, d["w_gate_up"], d["w_down"])[0]
    lg[1] = float("nan")
    out, ids, _, ws = moe.fwd_few_logits(d["hidden"], lg, 2, d["w_gate_up"], d["w_down"])
    assert torch.all(ids[1] == -1) and torch.all(out[1] == 0)
    assert torch.equal(out[[0, 2]], ref[[0, 2]])
    assert moe.check_device_status(ws) == moe.MOE_ERR_BAD_EXPERT_ID


def test_agrees_with_the_forward():
    """fwd_few and fwd compute one layer: both within the bound of it."""
    inp = small_inputs(24, 320, 192, 8, 2, "bf16", "clamped", "interleaved", seed=11)
    got, _ = run_case(inp)
    d = device_inputs(inp)
    full, _, _ = moe.fwd(d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"], act="clamped",
                         layout="interleaved")
    ref, bound = layer_bound(inp.hidden, inp.topk_ids, inp.topk_weights, list(zip(inp.w_gate_up, inp.w_down)), "clamped",
                             "interleaved", "bf16")
    check_layer(host(full), ref, bound)


def test_side_stream_and_capture():
    """On a stream of its own, and captured once and replayed on new inputs, with eager calls between."""
    a, b = (small_inputs(6, 136, 72, 40, 2, "bf16", "swiglu", "concat", seed=s) for s in (1, 2))
    d = device_inputs(a)
    want = [moe.fwd_few(x["hidden"], x["topk_ids"], x["topk_weights"], d["w_gate_up"], d["w_down"])[0]
            for x in (device_inputs(a), device_inputs(b))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, ws = moe.fwd_few(d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"])
    s.synchronize()
    assert torch.equal(out, want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.fwd_few(d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"], ws=ws, out=out)
    for i in (1, 0, 1, 1, 0):
        x = device_inputs((a, b)[i])
        for n in ("hidden", "topk_ids", "topk_weights"):
            d[n].copy_(x[n])
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        eager, _ = moe.fwd_few(d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"])
        assert torch.equal(eager, want[i])


def test_full_size_layer():
    """The gpt-oss-shaped layer: 9 tokens on few experts (rows of 2880, weights past 2^31 bytes from the base)."""
    T, H, I, E, K = 9, 2880, 2880, 70, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    gu = torch.randn((E, 2 * I, H), generator=g, device="cuda", dtype=torch.bfloat16).mul_(0.02)
    dn = torch.randn((E, H, I), generator=g, device="cuda", dtype=torch.bfloat16).mul_(0.02)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    ids = torch.tensor([[0, 1, 69, 68]] * 5 + [[69, 3, 1, 2]] * 4, dtype=torch.int32, device="cuda")
    w = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1)
    out, _ = moe.fwd_few(x, ids, w, gu, dn, act="clamped", layout="interleaved")
    used = {e: (host(gu[e]), host(dn[e])) for e in (0, 1, 2, 3, 68, 69)}
    none = (np.zeros((2 * I, 1)), np.zeros((1, I)))
    ref, bound = layer_bound(host(x), ids.cpu().numpy(), host(w), [used.get(e, none) for e in range(E)], "clamped", "interleaved",
                             "bf16")
    check_layer(host(out), ref, bound)


def test_two_streams_at_once():
    """Calls that overlap on two streams, with workspaces of their own."""
    cases = [small_inputs(T, 512, 256, 16, 4, "bf16", "swiglu", "concat", seed=T) for T in (3, 40)]
    dev = [device_inputs(c) for c in cases]
    args = [(d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"]) for d in dev]
    want = [moe.fwd_few(*a)[0] for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(moe.fwd_few(*args[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_refusals_of_the_binding():
    inp = small_inputs(4, 64, 32, 4, 2, "bf16", "swiglu", "concat")
    d = device_inputs(inp)
    x, ids, w, gu, dn = d["hidden"], d["topk_ids"], d["topk_weights"], d["w_gate_up"], d["w_down"]
    for bad in [(x.t().contiguous().t(), ids, w, gu, dn), (x.float(), ids, w, gu, dn), (x.half(), ids, w, gu.half(), dn.half()),
                (x, ids, w, gu[:, :, :32], dn), (x, ids[:2], w, gu, dn), (x, ids, w[:, :1], gu, dn),
                (x, ids, w, gu.transpose(1, 2), dn), (x, ids.cpu(), w, gu, dn), (x, ids, w, gu, dn.cpu()), (x[0], ids, w, gu, dn)]:
        with pytest.raises(ValueError):
            moe.fwd_few(*bad)
    for kw in (dict(act="gelu"), dict(layout="rows"), dict(out=torch.empty(4, 64, device="cuda")),
               dict(out=torch.empty(4, 64, dtype=torch.bfloat16)), dict(ws=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            moe.fwd_few(x, ids, w, gu, dn, **kw)
    with pytest.raises(moe.MoeError) as e:
        moe.fwd_few(x, ids, w, gu, dn, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == moe.MOE_ERR_WORKSPACE
    many = torch.zeros(129, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError) as e:
        moe.fwd_few(many, torch.zeros(129, 2, dtype=torch.int32, device="cuda"), torch.ones(129, 2, device="cuda"), gu, dn)
    assert e.value.status == moe.MOE_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        moe.fwd_few_logits(x, torch.zeros(4, 5, device="cuda"), 2, gu, dn)
    with pytest.raises(moe.MoeError) as e:
        moe.fwd_few_logits(x, torch.zeros(4, 4, device="cuda"), 5, gu, dn)
    assert e.value.status == moe.MOE_ERR_INVALID_ARG


def test_other_id_and_weight_types():
    """64-bit ids and half-precision weights are converted; an out tensor of the caller's is filled."""
    inp = small_inputs(4, 64, 32, 4, 2, "bf16", "swiglu", "concat")
    d = device_inputs(inp)
    want, _ = moe.fwd_few(d["hidden"], d["topk_ids"], d["topk_weights"].bfloat16().float(), d["w_gate_up"], d["w_down"])
    out = torch.empty_like(want)
    got, _ = moe.fwd_few(d["hidden"], d["topk_ids"].long(), d["topk_weights"].bfloat16(), d["w_gate_up"], d["w_down"], out=out)
    assert got is out and torch.equal(got, want)
