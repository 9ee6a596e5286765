"""The norms around a block, the step between them, and their backward passes against 64 bits."""
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
from tests._block import E, SECOND, STAT, Norm, check, column_sum, half_step

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rand(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dt).cuda()


def inputs(T, H, dtype, gate="row", post=True, nxt=True, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    d = dict(x=rand(g, (T, H), dt, std), h=rand(g, (T, H), dt, 0.5 * std), dx=rand(g, (T, H), dt), dy=rand(g, (T, H), dt) if nxt else None,
             w_post=1 + rand(g, (H,), dt, 0.2) if post else None, w_next=1 + rand(g, (H,), dt, 0.2) if nxt else None)
    shape = {"none": None, "row": (T, 1), "column": (H,), "full": (T, H)}[gate]
    d["gate"] = None if shape is None else rand(g, shape, dt)
    return d


def nan_like(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def residual_case(d, gate, scale=0.7, eps=1e-5):
    x, h, dt = d["x"], d["h"], d["x"].dtype
    u = half_step(dt)
    kw = dict(w_post=d["w_post"], gate=d["gate"], scale=scale, w_next=d["w_next"], eps=eps)
    new, y = moe.residual_fwd(x, h, x_new=nan_like(x.shape, dt), y=nan_like(x.shape, dt) if d["w_next"] is not None else None, **kw)
    post = Norm(h, d["w_post"], eps) if d["w_post"] is not None else None
    n, en = (post.n, post.en) if post else (h.double(), 0 * h.double())
    f = torch.full((), scale, dtype=torch.float32).double().to(x.device)   # the scale as the call takes it
    gt = d["gate"].double() if d["gate"] is not None else torch.ones((), dtype=torch.float64, device=x.device)
    ref = x.double() + f * gt * n
    err = (f * gt).abs() * (en + 4 * E * n.abs()) + 2 * E * ref.abs()
    check(new, ref, SECOND * (err + u * ref.abs()), "x_new")
    if d["w_next"] is None:
        assert y is None
    else:
        nx = Norm(ref, d["w_next"], eps)
        _, ey, _, _ = nx.grad(torch.zeros_like(ref))
        # x_new's error passes through the norm: r w (e - hat mean(hat e))
        through = nx.r * nx.w.abs() * (err + nx.hat.abs() * (nx.hat.abs() * err).mean(-1, keepdim=True))
        check(y, nx.n, SECOND * (through + nx.en + u * nx.n.abs()), "y")
    # backward, on x_new as it was stored
    grads = moe.ResidualGrads(nan_like(x.shape, dt), nan_like(x.shape, dt),
                              nan_like(d["gate"].shape, dt if gate == "full" else torch.float32) if gate != "none" else None,
                              nan_like(x.shape[1:], torch.float32), nan_like(x.shape[1:], torch.float32), None)
    got = moe.residual_bwd(new, h, d["dx"], d["dy"], grads=grads, **kw)
    t, et = d["dx"].double(), 0 * d["dx"].double()
    if d["w_next"] is not None:
        nx = Norm(new, d["w_next"], eps)
        dv, ev, tn, etn = nx.grad(d["dy"].double())
        t, et = t + dv, ev + 2 * E * (t.abs() + dv.abs())
        check(got.d_w_next, *column_sum(tn, etn), "d_w_next")
    check(got.d_x, t, SECOND * (et + u * t.abs()), "d_x")
    dn, edn = f * gt * t, (f * gt).abs() * (et + 4 * E * t.abs())
    if post:
        dh, edh, tp, etp = post.grad(dn, edn)
        check(got.d_w_post, *column_sum(tp, etp), "d_w_post")
    else:
        dh, edh = dn, edn
        assert got.d_w_post is None
    check(got.d_h, dh, SECOND * (edh + u * dh.abs()), "d_h")
    terms, eterms = f * t * n, abs(scale) * (et * n.abs() + t.abs() * en + 6 * E * (t * n).abs())
    if gate == "row":
        check(got.d_gate, terms.sum(1, keepdim=True), SECOND * (eterms + STAT * terms.abs()).sum(1, keepdim=True), "d_gate")
    elif gate == "column":
        check(got.d_gate, *column_sum(terms, eterms), "d_gate")
    elif gate == "full":
        check(got.d_gate, terms, SECOND * (eterms + u * terms.abs()), "d_gate")
    else:
        assert got.d_gate is None
    return new, y, got


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gate", ["none", "row", "column", "full"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("nxt", [True, False])
def test_parts(dtype, gate, post, nxt):
    residual_case(inputs(37, 264, dtype, gate, post, nxt, seed=4), gate)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H", [8, 16, 504, 512, 520, 1024, 1032, 2880, 4096, 4104, 8192, 8200, 16384])
def test_row_lengths(H, dtype):
    residual_case(inputs(11, H, dtype, "column", seed=H), "column")
    residual_case(inputs(3, H, dtype, "full", seed=H + 1), "full")


@pytest.mark.parametrize("gate", ["row", "column", "none"])
@pytest.mark.parametrize("T", [1, 2, 511, 512, 513, 1500, 5000])
def test_row_counts(T, gate):
    residual_case(inputs(T, 72, "bf16", gate, seed=T), gate)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 520), (700, 264), (1, 16384), (600, 2880)])
def test_before_a_block(T, H, dtype):
    d = inputs(T, H, dtype, seed=T + H)
    x, w, dt = d["x"], d["w_next"], d["x"].dtype
    u = half_step(dt)
    ref = Norm(x, w, 1e-5)
    check(moe.norm_fwd(x, w, out=nan_like(x.shape, dt)), ref.n, SECOND * (ref.en + u * ref.n.abs()), "y")
    g, eg, t, et = ref.grad(d["dy"].double())
    for add in (d["dx"], None):
        dx, dw, _ = moe.norm_bwd(x, w, d["dy"], d_add=add, grads=(nan_like(x.shape, dt), nan_like((H,), torch.float32)))
        want = g + (add.double() if add is not None else 0.0)
        check(dx, want, SECOND * (eg + 2 * E * (g.abs() + want.abs()) + u * want.abs()), "d_x")
        check(dw, *column_sum(t, et), "d_w")
    step = moe.residual_bwd(x, d["h"], d["dx"], d["dy"], w_next=w)
    assert torch.equal(step.d_x, moe.norm_bwd(x, w, d["dy"], d_add=d["dx"])[0])


def test_large_and_small_values():
    """Squares of values around 1e15 and 1e-15 stay in fp32's range; a zero row gives zeros, its gradients are finite."""
    for std in (1e15, 1e-15):
        d = inputs(9, 200, "fp32", "row", seed=1, std=std)
        new, _ = moe.residual_fwd(d["x"], d["h"], scale=1.0)
        check(moe.norm_fwd(new, d["w_next"], eps=0.0), Norm(new, d["w_next"], 0.0).n, SECOND * 2 * STAT * Norm(new, d["w_next"], 0.0).n.abs())
    d = inputs(5, 64, "bf16", "row")
    d["x"][1] = 0
    d["h"][1] = 0
    new, y, got = residual_case(d, "row")
    assert not new[1].any() and not y[1].any()


def test_non_finite_rows_stay_rows():
    d = inputs(20, 136, "bf16", "row", seed=6)
    kw = dict(w_post=d["w_post"], gate=d["gate"], w_next=d["w_next"])
    x0, y0 = moe.residual_fwd(d["x"], d["h"], **kw)
    d["h"][3, 7], d["x"][5, 1] = float("nan"), float("inf")
    x1, y1 = moe.residual_fwd(d["x"], d["h"], **kw)
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[3] = keep[5] = False
    assert torch.equal(x0[keep], x1[keep]) and torch.equal(y0[keep], y1[keep])
    assert torch.isnan(y1[3]).all() and torch.isinf(x1[5, 1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_in_place_and_nothing_behind(dtype):
    d = inputs(21, 136, dtype, "row", seed=7)
    kw = dict(w_post=d["w_post"], gate=d["gate"], w_next=d["w_next"])
    new, y = moe.residual_fwd(d["x"], d["h"], **kw)
    want = moe.residual_bwd(new, d["h"], d["dx"], d["dy"], **kw)
    big = torch.full((40, 136), 3.0, dtype=d["x"].dtype, device="cuda")
    big[:21] = d["x"]
    moe.residual_fwd(big[:21], d["h"], x_new=big[:21], **kw)
    assert torch.equal(big[:21], new) and bool((big[21:] == 3).all())
    big[:21] = d["dx"]
    moe.residual_bwd(new, d["h"], big[:21], d["dy"], grads=moe.ResidualGrads(big[:21], None, None, None, None, None), **kw)
    assert torch.equal(big[:21], want.d_x) and bool((big[21:] == 3).all())
    big[:21] = d["dx"]
    moe.norm_bwd(new, d["w_next"], d["dy"], d_add=big[:21], grads=(big[:21], None))
    assert torch.equal(big[:21], want.d_x)


@pytest.mark.parametrize("gate", ["none", "column"])
def test_no_rows(gate):
    d = inputs(0, 64, "bf16", gate)
    new, y = moe.residual_fwd(d["x"], d["h"], w_post=d["w_post"], gate=d["gate"], w_next=d["w_next"])
    assert new.shape == y.shape == (0, 64)
    got = moe.residual_bwd(new, d["h"], d["dx"], d["dy"], w_post=d["w_post"], gate=d["gate"], w_next=d["w_next"],
                           grads=moe.ResidualGrads(None, None, nan_like((64,), torch.float32) if gate == "column" else None,
                                                   nan_like((64,), torch.float32), nan_like((64,), torch.float32), None))
    assert not got.d_w_post.any() and not got.d_w_next.any() and (gate == "none" or not got.d_gate.any())
    _, dw, _ = moe.norm_bwd(d["x"], d["w_next"], d["dy"], grads=(None, nan_like((64,), torch.float32)))
    assert not dw.any()


def test_captured_and_replayed():
    d = inputs(700, 264, "bf16", "column", seed=3)
    kw = dict(w_post=d["w_post"], gate=d["gate"], w_next=d["w_next"])
    x = d["x"]
    new, y = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(moe.norm_workspace_size(moe._lib.NormDesc(700, 264, 0, 2, 1.0, 1e-5)), dtype=torch.uint8, device="cuda")
    f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    grads = moe.ResidualGrads(torch.empty_like(x), torch.empty_like(x), f(264), f(264), f(264), None)

    def step():
        moe.residual_fwd(x, d["h"], x_new=new, y=y, **kw)
        moe.residual_bwd(new, d["h"], d["dx"], d["dy"], ws=ws, grads=grads, **kw)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x.copy_(torch.randn(700, 264, generator=torch.Generator().manual_seed(k)).to(x.dtype))
        enew, ey = moe.residual_fwd(x, d["h"], **kw)
        want = moe.residual_bwd(enew, d["h"], d["dx"], d["dy"], **kw)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(new, enew) and torch.equal(y, ey)
        for a, b in zip(grads[:5], want[:5]):
            assert torch.equal(a, b)


def test_more_rows_than_one_dimension_of_a_launch():
    T, H = (1 << 26) + 5, 8   # 64 threads a row: over 2^32 threads
    x = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(9)).bfloat16()
    w = torch.linspace(0.5, 1.5, H, device="cuda").bfloat16()
    y = moe.norm_fwd(x, w, out=torch.full_like(x, float("nan")))
    for t0 in range(0, T, 1 << 24):
        n = Norm(x[t0:t0 + (1 << 24)], w, 1e-5)
        check(y[t0:t0 + (1 << 24)], n.n, SECOND * (n.en + half_step(torch.bfloat16) * n.n.abs()), "y")


@pytest.mark.parametrize("gate", ["none", "row", "column", "full"])
@pytest.mark.parametrize("T,H", [(513, 1032), (1025, 2048), (700, 512), (1537, 1024), (2051, 8), (1300, 2056)])
def test_short_rows_share_workgroups(T, H, gate):
    """Rows that do not fill the last workgroup of several, at one and two waves a row and past them."""
    for dtype in TYPES:
        residual_case(inputs(T, H, dtype, gate, seed=T + H), gate)
