"""4-bit microscaled weights: the format bit for bit, and the layer on them against 64 bits."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
from tests._gpu import host, small_inputs
from tests._serve import check_layer, layer_bound, pack, quantize_ref, values_ref

pytestmark = pytest.mark.gpu


def check_rows(w):
    """mx_quantize of a device tensor against the definition, and mx_dequantize of the result."""
    codes, scales = moe.mx_quantize(w)
    x = w.float().cpu().numpy()
    rc, rs = quantize_ref(x)
    assert np.array_equal(scales.cpu().numpy().reshape(-1), rs)
    assert np.array_equal(codes.cpu().numpy().reshape(-1, 16), pack(rc))
    want = values_ref(codes.cpu().numpy(), scales.cpu().numpy())
    for dtype in ("bf16", "fp32"):
        got = moe.mx_dequantize(codes, scales, dtype=dtype)
        assert got.shape == w.shape
        assert np.array_equal(host(got).astype(np.float64), want, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 32), (3, 32), (1, 64), (7, 96), (5, 736), (33, 1056), (2, 3, 160), (1, 8224)])
def test_random_rows(dtype, shape):
    w = torch.randn(shape, generator=torch.Generator().manual_seed(shape[0])).to(dtype).cuda()
    check_rows(0.02 * w)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_and_ends_of_every_binade(dtype):
    """Each block: its largest magnitude at a binade's start or end, and the rounding borders below it."""
    marks = [0, 0.25, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.9375, 0.2490234375, 0.2509765625, 4.96875, 5.03125]
    rows = []
    for ex in (-133, -130, -127, -126, -125, -124, -100, -8, 0, 1, 60, 100, 124, 125):
        for top in (4.0, 5.0, 7.9375):
            b = np.array(marks + [-m for m in marks]) * 2.0 ** ex
            b[np.abs(b) > top * 2.0 ** ex] = 0
            b[0] = top * 2.0 ** ex
            rows.append(b)
    with np.errstate(over="ignore"):
        w = torch.tensor(np.array(rows)).to(torch.float32).to(dtype).cuda()
    check_rows(w)


def test_every_bf16_value():
    """All 65536 bit patterns, 31 of them to a block behind a fixed largest element, and in blocks of neighbours."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    check_rows(v.reshape(-1, 32).cuda())
    small = v[torch.isfinite(v.float()) & (v.float().abs() <= 6.0)]
    small = small[: len(small) // 31 * 31].reshape(-1, 31)
    check_rows(torch.cat((torch.full((len(small), 1), 6.0, dtype=torch.bfloat16), small), dim=1).contiguous().cuda())


def test_non_finite_blocks():
    w = torch.randn(6, 96, generator=torch.Generator().manual_seed(0))
    w[0, 3], w[1, 40], w[2, 95], w[4, 0] = float("nan"), float("inf"), float("-inf"), float("nan")
    w[5] = 0
    w[5, 1] = -0.0
    for dtype in (torch.bfloat16, torch.float32):
        check_rows(w.to(dtype).cuda())


def test_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).reshape(16, 16).repeat(256, 1).cuda()
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(16).reshape(-1, 1).contiguous().cuda()
    want = values_ref(codes.cpu().numpy(), scales.cpu().numpy())
    for dtype in ("bf16", "fp32"):
        got = host(moe.mx_dequantize(codes, scales, dtype=dtype)).astype(np.float64)
        with np.errstate(over="ignore"):
            w32 = want.astype(np.float32).astype(np.float64)   # 2^127 times 2 and more is past both types' range
        assert np.array_equal(got, w32, equal_nan=True)


def test_large_rows_run_in_a_loop():
    """More elements than one pass of the largest grid would hold per thread, on a capped row count."""
    n = 1 << 22
    w = torch.randn((n // 2048, 2048), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    codes, scales = moe.mx_quantize(w)
    v = moe.mx_dequantize(codes, scales, dtype="fp32")
    pick = torch.randint(0, n // 2048, (64,), generator=torch.Generator().manual_seed(2))
    rc, rs = quantize_ref(w[pick].cpu().numpy())
    assert np.array_equal(codes[pick].cpu().numpy().reshape(-1, 16), pack(rc))
    assert np.array_equal(scales[pick].cpu().numpy().reshape(-1), rs)
    assert torch.equal(moe.mx_dequantize(codes[pick].contiguous(), scales[pick].contiguous(), dtype="fp32"), v[pick])


def mx_case(inp, poison=True):
    """mx_fwd on the quantised weights of inp, poisoned buffers, against 64 bits on the dequantised ones."""
    wl = inp.wl
    gu = moe.mx_quantize(torch.from_numpy(inp.w_gate_up).cuda())
    dn = moe.mx_quantize(torch.from_numpy(inp.w_down).cuda())
    x = torch.from_numpy(inp.hidden).cuda().bfloat16()
    ids, w = torch.from_numpy(inp.topk_ids).cuda(), torch.from_numpy(inp.topk_weights).cuda()
    desc = moe.make_desc(wl.T, wl.H, wl.I, wl.E, ids.shape[1], "bf16", wl.act, wl.layout)
    ws = torch.full((moe.mx_workspace_size(desc),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(x, float("nan"))
    kw = dict(act=wl.act, layout=wl.layout)
    got, _ = moe.mx_fwd(x, ids, w, gu, dn, ws=ws, out=out, **kw)
    again, _ = moe.mx_fwd(x, ids, w, gu, dn, **kw)
    torch.cuda.synchronize()
    assert torch.equal(got, again)
    vg, vd = (values_ref(q[0].cpu().numpy(), q[1].cpu().numpy()) for q in (gu, dn))
    ref, bound = layer_bound(inp.hidden, inp.topk_ids, inp.topk_weights, list(zip(vg, vd)), wl.act, wl.layout, "bf16")
    check_layer(host(got), ref, bound, wl.name)
    return got, ws


TOKENS = [1, 2, 15, 16, 17, 33, 128, 129, 200, 513]


@pytest.mark.parametrize("T", TOKENS)
def test_token_counts(T):
    mx_case(small_inputs(T, 160, 96, 7, 2, "bf16", "clamped", "interleaved", seed=T))


@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("H,I", [(32, 32), (64, 32), (32, 96), (288, 128), (256, 320), (1056, 736), (96, 1120)])
def test_sizes(T, H, I):
    mx_case(small_inputs(T, H, I, 5, 3, "bf16", "swiglu", "concat", seed=H + I))


@pytest.mark.parametrize("T", [9, 260])
@pytest.mark.parametrize("act", ["swiglu", "clamped"])
@pytest.mark.parametrize("layout", ["concat", "interleaved"])
def test_activation_and_layout(T, act, layout):
    mx_case(small_inputs(T, 192, 160, 4, 2, "bf16", act, layout, seed=3, xscale=8.0))


@pytest.mark.parametrize("T,E,K", [(4, 1, 1), (300, 1, 1), (4, 200, 8), (140, 200, 8), (130, 1024, 2), (3, 64, 64), (140, 64, 64)])
def test_expert_counts(T, E, K):
    mx_case(small_inputs(T, 64, 32, E, K, "bf16", "swiglu", "interleaved", seed=E))


@pytest.mark.parametrize("T", [16, 33, 128, 129, 256, 257, 300, 700])
def test_one_expert_takes_every_token(T):
    ids = np.full((T, 1), 2, dtype=np.int32)
    mx_case(small_inputs(T, 288, 160, 4, 1, "bf16", "clamped", "concat", seed=T, ids=ids))


@pytest.mark.parametrize("T", [32, 33, 128])
def test_large_layer_of_few_experts(T):
    mx_case(small_inputs(T, 1472, 1472, 2, 2, "bf16", "swiglu", "concat", seed=T))


@pytest.mark.parametrize("T,H,E,K", [(125, 2304, 3, 3), (128, 2304, 3, 3), (64, 160, 2, 2), (65, 160, 2, 2), (128, 96, 3, 3)])
def test_sides_of_the_rule_of_many_slots(T, H, E, K):
    """S H I just below and above 2e9, and 64 slots an expert and more: the latter run the grouped products."""
    mx_case(small_inputs(T, H, H, E, K, "bf16", "clamped", "interleaved", seed=T + H))


@pytest.mark.parametrize("T", [3, 140])
def test_long_rows(T):
    """Rows of many scales: past the few-token kernels' limit of 8192, and the longest ones."""
    for H, I in ((8224, 32), (32, 8224), (14336, 32), (32, 14336)):
        mx_case(small_inputs(T, H, I, 2, 1, "bf16", "swiglu", "interleaved", seed=T))


@pytest.mark.parametrize("K", [1, 2, 3, 5, 8, 9, 17, 64])
def test_one_token(K):
    """One token's own kernels: fewer, as many and more slots than waves."""
    mx_case(small_inputs(1, 288, 160, 64, K, "bf16", "clamped", "interleaved", seed=K))
    mx_case(small_inputs(1, 160, 288, 64, K, "bf16", "swiglu", "concat", seed=K))
    ids = np.resize(np.array([3, -1, 3, 64, 5], dtype=np.int32), (1, K))
    got, ws = mx_case(small_inputs(1, 96, 64, 64, K, "bf16", "swiglu", "concat", seed=K, ids=ids))
    assert moe.check_device_status(ws) == (moe.MOE_ERR_BAD_EXPERT_ID if K > 1 else moe.MOE_OK)


def test_most_slots_and_long_rows():
    """128 tokens of 64 slots on rows of 8192: the few-token kernels' LDS would not hold them."""
    mx_case(small_inputs(128, 8192, 32, 256, 64, "bf16", "swiglu", "concat", seed=1))


@pytest.mark.parametrize("T", [20, 150])
def test_non_finite_tokens_stay_alone(T):
    H, I, E = 160, 96, 5
    ids = np.stack((np.arange(T) % E, (np.arange(T) + 1) % E), axis=1).astype(np.int32)
    inp = small_inputs(T, H, I, E, 2, "bf16", "swiglu", "concat", seed=T, ids=ids)
    gu, dn = (moe.mx_quantize(torch.from_numpy(v).cuda()) for v in (inp.w_gate_up, inp.w_down))
    x, w = torch.from_numpy(inp.hidden).cuda().bfloat16(), torch.from_numpy(inp.topk_weights).cuda()
    i = torch.from_numpy(ids).cuda()
    want, _ = moe.mx_fwd(x, i, w, gu, dn)
    x[3], x[T - 1, 5], w[7, 1] = float("nan"), float("inf"), float("inf")
    got, _ = moe.mx_fwd(x, i, w, gu, dn)
    assert torch.all(torch.isnan(got[3])) and not torch.any(torch.isfinite(got[7])) and not torch.all(torch.isfinite(got[T - 1]))
    rest = [t for t in range(T) if t not in (3, 7, T - 1)]
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("T", [4, 200])
def test_bad_ids_are_dropped_and_reported(T):
    E = 5
    rows = np.array([[0, -1, 2], [E, E + 7, -(2 ** 31)], [2 ** 31 - 1, 4, 4], [1, 2, 3]], dtype=np.int32)
    ids = np.tile(rows, (T // 4, 1))
    got, ws = mx_case(small_inputs(T, 96, 64, E, 3, "bf16", "swiglu", "concat", seed=4, ids=ids))
    assert moe.check_device_status(ws) == moe.MOE_ERR_BAD_EXPERT_ID
    assert torch.all(got[1::4] == 0)
    assert moe.check_device_status(mx_case(small_inputs(T, 96, 64, E, 3, "bf16", "swiglu", "concat", seed=4))[1]) == moe.MOE_OK


@pytest.mark.parametrize("T", [2, 140])
def test_nan_scales_stay_with_their_expert(T):
    """A NaN block reaches every token of its expert and no other; scale bytes 0 and 254 are ordinary."""
    H, I, E = 160, 96, 4
    g = torch.Generator().manual_seed(T)
    gu = [torch.randint(0, 256, (E, 2 * I, H // 2), dtype=torch.uint8, generator=g),
          torch.randint(116, 122, (E, 2 * I, H // 32), dtype=torch.uint8, generator=g)]
    dn = [torch.randint(0, 256, (E, H, I // 2), dtype=torch.uint8, generator=g),
          torch.randint(116, 122, (E, H, I // 32), dtype=torch.uint8, generator=g)]
    gu[1][0, 5, :] = 0           # a row of 2^-127
    dn[1][3, :, 1] = 255
    ids = (torch.arange(T) % E).to(torch.int32).reshape(T, 1)
    x, w = torch.randn(T, H, generator=g).bfloat16(), torch.ones(T, 1)
    out, _ = moe.mx_fwd(x.cuda(), ids.cuda(), w.cuda(), [t.cuda() for t in gu], [t.cuda() for t in dn])
    out = host(out)
    bad = ids[:, 0].numpy() == 3
    assert np.all(np.isnan(out[bad]))
    vg, vd = (values_ref(q[0].numpy(), q[1].numpy()) for q in (gu, dn))
    ref, bound = layer_bound(x.float().numpy()[~bad], ids.numpy()[~bad], w.numpy()[~bad], list(zip(vg, vd))[:3], "swiglu", "concat",
                             "bf16")
    check_layer(out[~bad], ref, bound)


@pytest.mark.parametrize("T,E,K", [(1, 128, 4), (16, 33, 8), (150, 9, 2)])
def test_from_logits(T, E, K):
    inp = small_inputs(T, 64, 64, E, K, "bf16", "clamped", "interleaved", seed=T)
    gu, dn = (moe.mx_quantize(torch.from_numpy(v).cuda()) for v in (inp.w_gate_up, inp.w_down))
    x = torch.from_numpy(inp.hidden).cuda().bfloat16()
    lg = torch.randn(T, E, generator=torch.Generator().manual_seed(T)).cuda()
    kw = dict(act="clamped", layout="interleaved")
    out, ids, w, ws = moe.mx_fwd_logits(x, lg, K, gu, dn, **kw)
    rids, rw = moe.router(lg, K)[:2]
    assert torch.equal(ids, rids) and torch.equal(w, rw)
    assert torch.equal(out, moe.mx_fwd(x, rids, rw, gu, dn, **kw)[0])
    assert moe.check_device_status(ws) == moe.MOE_OK


def test_no_tokens():
    q = (torch.zeros(2, 64, 32, dtype=torch.uint8, device="cuda"), torch.zeros(2, 64, 2, dtype=torch.uint8, device="cuda"))
    dq = (torch.zeros(2, 64, 16, dtype=torch.uint8, device="cuda"), torch.zeros(2, 64, 1, dtype=torch.uint8, device="cuda"))
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    out, ws = moe.mx_fwd(x, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, 2, device="cuda"), q, dq)
    assert tuple(out.shape) == (0, 64) and moe.check_device_status(ws) == moe.MOE_OK
    c, s = moe.mx_quantize(torch.zeros(0, 64, device="cuda"))
    assert tuple(c.shape) == (0, 32) and tuple(s.shape) == (0, 2)


@pytest.mark.parametrize("T", [3, 160])
def test_capture_and_replay(T):
    a, b = (small_inputs(T, 160, 96, 6, 2, "bf16", "swiglu", "concat", seed=s) for s in (1, 2))
    gu, dn = (moe.mx_quantize(torch.from_numpy(v).cuda()) for v in (a.w_gate_up, a.w_down))
    dev = [tuple(torch.from_numpy(v).cuda() for v in (i.hidden, i.topk_ids, i.topk_weights)) for i in (a, b)]
    dev = [(x.bfloat16(), i, w) for x, i, w in dev]
    want = [moe.mx_fwd(*d, gu, dn)[0] for d in dev]
    cur = tuple(t.clone() for t in dev[0])
    out, ws = moe.mx_fwd(*cur, gu, dn)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.mx_fwd(*cur, gu, dn, ws=ws, out=out)
    for i in (1, 0, 1, 1, 0):
        for c, d in zip(cur, dev[i]):
            c.copy_(d)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        assert torch.equal(moe.mx_fwd(*cur, gu, dn)[0], want[i])


def test_quantise_route_and_decode_together():
    """As a server uses them: quantise bf16 experts once, run a prompt through the layer from router logits, then decode
    token by token on the same weights; each token's output is the prompt's, to rounding."""
    T, H, I, E, K = 150, 192, 96, 12, 3
    inp = small_inputs(T, H, I, E, K, "bf16", "clamped", "interleaved", seed=6)
    gu, dn = (moe.mx_quantize(torch.from_numpy(v).cuda().bfloat16()) for v in (inp.w_gate_up, inp.w_down))
    x = torch.from_numpy(inp.hidden).cuda().bfloat16()
    lg = torch.randn(T, E, generator=torch.Generator().manual_seed(8)).cuda()
    kw = dict(act="clamped", layout="interleaved")
    out, ids, w, ws = moe.mx_fwd_logits(x, lg, K, gu, dn, **kw)
    vg, vd = (values_ref(q[0].cpu().numpy(), q[1].cpu().numpy()) for q in (gu, dn))
    ref, bound = layer_bound(inp.hidden, ids.cpu().numpy(), host(w), list(zip(vg, vd)), "clamped", "interleaved", "bf16")
    check_layer(host(out), ref, bound)
    steps = torch.cat([moe.mx_fwd_logits(x[t:t + 1], lg[t:t + 1], K, gu, dn, **kw)[0] for t in range(0, T, 7)])
    check_layer(host(steps), ref[::7], bound[::7])
    # the same experts dequantised, through the few-token and the full forward
    dg, dd = moe.mx_dequantize(*gu), moe.mx_dequantize(*dn)
    check_layer(host(moe.fwd_few(x[:100], ids[:100], w[:100], dg, dd, **kw)[0]), ref[:100], bound[:100])
    check_layer(host(moe.fwd(x, ids, w, dg, dd, **kw)[0]), ref, bound)


def test_rows_past_the_output_stay():
    """A call of T tokens into the first rows of longer buffers leaves the rest as it was."""
    for T in (1, 5, 150):
        inp = small_inputs(T, 96, 64, 4, 2, "bf16", "swiglu", "concat", seed=T)
        gu, dn = (moe.mx_quantize(torch.from_numpy(v).cuda()) for v in (inp.w_gate_up, inp.w_down))
        x = torch.from_numpy(inp.hidden).cuda().bfloat16()
        ids, w = torch.from_numpy(inp.topk_ids).cuda(), torch.from_numpy(inp.topk_weights).cuda()
        big = torch.full((T + 40, 96), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.mx_fwd(x, ids, w, gu, dn, out=big[:T])
        assert torch.all(big[T:] == 7) and torch.equal(big[:T], moe.mx_fwd(x, ids, w, gu, dn)[0])


def test_quantize_into_the_callers_buffers():
    w = torch.randn(6, 160, generator=torch.Generator().manual_seed(3)).cuda()
    codes, scales = moe.mx_quantize(w)
    pc = torch.full((10, 80), 0xEE, dtype=torch.uint8, device="cuda")
    ps = torch.full((10, 5), 0xEE, dtype=torch.uint8, device="cuda")
    moe.mx_quantize(w, out=(pc[:6], ps[:6]))
    assert torch.equal(pc[:6], codes) and torch.equal(ps[:6], scales)
    assert torch.all(pc[6:] == 0xEE) and torch.all(ps[6:] == 0xEE)
    v = torch.full((8, 160), 7.0, device="cuda")
    moe.mx_dequantize(codes, scales, dtype="fp32", out=v[:6])
    assert torch.equal(v[:6], moe.mx_dequantize(codes, scales, dtype="fp32")) and torch.all(v[6:] == 7)


def test_refusals_of_the_binding():
    w = torch.randn(4, 96, device="cuda")
    for bad in (w.t(), w[:, :48].contiguous(), w.half(), w[:, 0:0]):
        with pytest.raises(ValueError):
            moe.mx_quantize(bad)
    with pytest.raises(moe.MoeError):
        moe.mx_quantize(torch.randn(4 * 96 + 1, device="cuda")[1:].reshape(4, 96))   # not 16-byte aligned
    codes, scales = moe.mx_quantize(w)
    for c, s in ((codes, scales[:, :2]), (codes[:, :8], scales), (codes.int(), scales), (codes, scales.cpu())):
        with pytest.raises(ValueError):
            moe.mx_dequantize(c, s)
    with pytest.raises(ValueError):
        moe.mx_dequantize(codes, scales, dtype="fp16")
    inp = small_inputs(4, 64, 32, 4, 2, "bf16", "swiglu", "concat")
    gu, dn = (moe.mx_quantize(torch.from_numpy(v).cuda()) for v in (inp.w_gate_up, inp.w_down))
    x = torch.from_numpy(inp.hidden).cuda().bfloat16()
    ids, wt = torch.from_numpy(inp.topk_ids).cuda(), torch.from_numpy(inp.topk_weights).cuda()
    for bad in [(x.float(), ids, wt, gu, dn), (x, ids, wt, dn, gu), (x, ids, wt, (gu[0], dn[1]), dn), (x, ids[:1], wt, gu, dn),
                (x, ids, wt, (gu[0].to(torch.int8), gu[1]), dn)]:
        with pytest.raises(ValueError):
            moe.mx_fwd(*bad)
    with pytest.raises(moe.MoeError) as e:
        moe.mx_fwd(x, ids, wt, gu, dn, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == moe.MOE_ERR_WORKSPACE


def test_two_streams_at_once():
    """A prompt and a decode step on two streams, on the same weights."""
    inps = [small_inputs(T, 256, 160, 8, 2, "bf16", "swiglu", "concat", seed=1) for T in (2, 300)]
    gu, dn = (moe.mx_quantize(torch.from_numpy(v).cuda()) for v in (inps[0].w_gate_up, inps[0].w_down))
    args = [(torch.from_numpy(i.hidden).cuda().bfloat16(), torch.from_numpy(i.topk_ids).cuda(),
             torch.from_numpy(i.topk_weights).cuda(), gu, dn) for i in inps]
    want = [moe.mx_fwd(*a)[0] for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(moe.mx_fwd(*args[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])
