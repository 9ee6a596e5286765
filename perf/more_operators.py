"""Cases of the operators around the routed experts, with their plain forms.

Three operators of a mixture-of-experts block and its training step:

* "ffn":   the gated feed-forward block that every token passes beside its routed experts (the shared expert), or a dense
           layer's:  out[t] = add[t] + sigmoid(gate[t]) Wd phi(Wgu x_t), and its backward pass;
* "norm":  the norm before a block,  y = w x / rms(x),  and the step after it,
           x' = x + scale gate (w_post h / rms(h)),  y = w_next x' / rms(x'),  with their backward passes;
* "ortho": Newton-Schulz orthogonalisation of stacked weight updates,  X <- a X + b (X X^T) X + c (X X^T)^2 X  from
           X = G / |G|, alone or within an optimiser step (momentum, weight decay and the weights' update).

Layer sizes are those of the repository's workloads (H = I = 2880, E = 128, gate_up rows 5760; H = 4096, I = 2048) and
small ragged ones.  `own` selects the framework's calls; otherwise the operators are computed by elementary torch
operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

CLAMP, ALPHA = 7.0, 1.702
EPS = 1e-5                                    # of the norms
COEF, STEPS, TINY = (3.4445, -4.7750, 2.0315), 5, 1e-7
LR, MOMENTUM, DECAY = 0.02, 0.95, 0.002       # of the optimiser step: step size, momentum, step size times weight decay
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _ffn(name, T, H, I, act, layout, dtype="bf16", train=False, gated=True):
    return dict(name=name, op="ffn", T=T, H=H, I=I, act=act, layout=layout, dtype=dtype, train=train, gated=gated)


def _norm(name, T, H, dtype="bf16", train=False, after=True, gate="none", post=True):
    return dict(name=name, op="norm", T=T, H=H, dtype=dtype, train=train, after=after, gate=gate, post=post)


def _ortho(name, E, M, N, dtype="bf16", step=False):
    return dict(name=name, op="ortho", E=E, M=M, N=N, dtype=dtype, step=step)


def listed():
    return [
        # a decode step's shared expert for one chat, added to the routed experts' output
        _ffn("ffn 1 token", 1, 2880, 2880, "clamped", "interleaved"),
        # a small decode batch in fp32 at odd sizes: latency
        _ffn("ffn 13 tokens fp32 ragged", 13, 1048, 712, "swiglu", "concat", dtype="fp32"),
        # a prompt chunk through the shared expert
        _ffn("ffn 512 tokens", 512, 4096, 2048, "swiglu", "concat"),
        # the shared expert in training, at the repository's gpt-oss-shaped token count: forward and backward
        _ffn("ffn train 4096 tokens", 4096, 2880, 2880, "clamped", "interleaved", train=True),
        # a dense layer in training, no gate and nothing to add to
        _ffn("ffn train 8192 tokens wide", 8192, 4096, 8192, "swiglu", "concat", train=True, gated=False),
        # after a block and before the next in a decode batch: latency
        _norm("norm after, 16 tokens", 16, 2880, gate="row"),
        # before a block in training: forward, and backward with the residual's gradient added
        _norm("norm before, train 4096", 4096, 2880, train=True, after=False),
        # after a block in training: post-norm, a gate for each token, the next block's norm
        _norm("norm after, train 32768", 32768, 4096, train=True, gate="row"),
        # the same in fp32 with a learned gate for each channel, odd sizes
        _norm("norm after, train 1000 fp32", 1000, 1048, dtype="fp32", train=True, gate="column"),
        # the down projections of 16 experts, bf16 gradients
        _ortho("ortho 16 of 2880 x 2880", 16, 2880, 2880),
        # an optimiser step of 8 experts' gate_up projections from fp32 gradients
        _ortho("step 8 of 5760 x 2880", 8, 5760, 2880, dtype="fp32", step=True),
        # many small ragged matrices, wider than high
        _ortho("ortho 24 of 200 x 712", 24, 200, 712),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Sizes of the same operators, over the ranges between the listed cases."""
    op = rng.choice(["ffn", "ffn", "ffn", "norm", "norm", "ortho", "ortho"])
    if op == "ffn":
        H, I = 8 * _log(rng, 32, 512), 8 * _log(rng, 32, 1024)
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        train = dtype == "bf16" and rng.random() < 0.6
        T = min(_log(rng, 1, 64) if dtype == "fp32" else _log(rng, 64 if train else 1, 8192), (8192 * 4096 * 8192) // (H * I))
        c = _ffn("", T, H, I, rng.choice(["swiglu", "clamped"]), rng.choice(["concat", "interleaved"]), dtype, train,
                 gated=rng.random() < 0.7)
    elif op == "norm":
        H, after = 8 * _log(rng, 32, 1024), rng.random() < 0.7
        T = min(_log(rng, 1, 32768), (32768 * 4096) // H)
        c = _norm("", T, H, rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.6, after,
                  rng.choice(["none", "row", "column", "full"]) if after else "none", rng.random() < 0.8 or not after)
    else:
        M, N = 8 * _log(rng, 12, 720), 8 * _log(rng, 12, 720)
        small, big = min(M, N), max(M, N)
        most = 8 * 2880 ** 2 * (4 * 5760 + 2 * 2880) // (small ** 2 * (4 * big + 2 * small))
        E = max(1, min(_log(rng, 1, 64), most))
        c = _ortho("", E, M, N, rng.choice(["bf16", "fp32"]), rng.random() < 0.4)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def rand(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    st = dict(case=case)
    if case["op"] == "ffn":
        # normed hidden states, weights of a trained layer's size, the routed experts' output, gate logits
        T, H, I = case["T"], case["H"], case["I"]
        st.update(x=rand(T, H), gu=rand(2 * I, H, std=0.02), dn=rand(H, I, std=0.02), gate=None, add=None)
        if case["gated"]:
            st.update(gate=rand(T, dtype=torch.float32), add=rand(T, H, std=0.5))
        if case["train"]:
            st["dout"] = rand(T, H, std=0.1)
    elif case["op"] == "norm":
        # a residual stream whose channels differ in size, a block's output, learned scales around one
        T, H = case["T"], case["H"]
        size = torch.exp(0.5 * torch.randn(H, generator=g, device=dev))
        st.update(x=(rand(T, H, dtype=torch.float32) * size).to(dt), w_next=(1 + rand(H, std=0.1, dtype=torch.float32)).to(dt),
                  h=None, w_post=None, gate=None, scale=1.0)
        if case["after"]:
            st.update(h=rand(T, H, std=0.3), scale=0.7)
            if case["post"]:
                st["w_post"] = (1 + rand(H, std=0.1, dtype=torch.float32)).to(dt)
            shape = {"none": None, "row": (T, 1), "column": (H,), "full": (T, H)}[case["gate"]]
            if shape:
                st["gate"] = torch.sigmoid(rand(*shape, dtype=torch.float32)).to(dt)
        if case["train"]:
            st.update(dx=rand(T, H, std=0.1), dy=rand(T, H, std=0.1))
    else:
        # gradients: a few strong directions over noise; weights and a momentum of the same kind
        E, M, N = case["E"], case["M"], case["N"]
        r = min(16, M, N)

        def update(dtype):
            s = torch.exp(-0.2 * torch.arange(r, device=dev))
            low = torch.bmm(torch.randn((E, M, r), generator=g, device=dev) * s, torch.randn((E, r, N), generator=g, device=dev))
            return (low.add_(torch.randn((E, M, N), generator=g, device=dev)).mul_(1e-4)).to(dtype)

        st["g"] = update(dt)
        if case["step"]:
            st.update(m=update(torch.float32).mul_(5), w=rand(E, M, N, std=0.02, dtype=torch.bfloat16))
    return st


# ------------------------------------------------------------------ the plain forms
def _halves(z, case):
    return (z[..., 0::2], z[..., 1::2]) if case["layout"] == "interleaved" else (z[..., :case["I"]], z[..., case["I"]:])


def _whole(dg, du, case):
    return torch.stack((dg, du), -1).flatten(-2) if case["layout"] == "interleaved" else torch.cat((dg, du), -1)


def _plain_ffn(st):
    case, dt = st["case"], st["x"].dtype
    x, gu, dn = st["x"].float(), st["gu"].float(), st["dn"].float()
    gate, up = _halves(x @ gu.t(), case)
    if case["act"] == "swiglu":
        sg = torch.sigmoid(gate)
        a = gate * sg * up
    else:
        gc, uc = gate.clamp(max=CLAMP), up.clamp(-CLAMP, CLAMP)
        sg = torch.sigmoid(ALPHA * gc)
        a = (uc + 1) * gc * sg
    y = a @ dn.t()
    s = torch.sigmoid(st["gate"])[:, None] if case["gated"] else 1.0
    out = (st["add"].float() + s * y if case["gated"] else y).to(dt)
    if not case["train"]:
        return dict(out=out)
    dout = st["dout"].float()
    r = dout @ dn
    da = s * r
    if case["act"] == "swiglu":
        dg, du = da * up * sg * (1 + gate * (1 - sg)), da * gate * sg
    else:
        dg = torch.where(gate <= CLAMP, da * (uc + 1) * sg * (1 + ALPHA * gc * (1 - sg)), 0.0)
        du = torch.where(uc == up, da * gc * sg, 0.0)
    dz = _whole(dg, du, case)
    got = dict(out=out, d_x=(dz @ gu).to(dt), d_gu=(dz.t() @ x).to(dt), d_dn=(dout.t() @ (s * a)).to(dt))
    if case["gated"]:
        got["d_gate"] = s[:, 0] * (1 - s[:, 0]) * (r * a).sum(1)
    return got


def _rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _norm_back(x, w, dy):
    """Gradients of w x / rms(x) with respect to x, and w row by row."""
    r = _rms(x)
    n, d = x * r, dy * w
    return r * (d - n * (d * n).mean(-1, keepdim=True)), dy * n


def _plain_norm(st):
    case, dt = st["case"], st["x"].dtype
    x, wn = st["x"].float(), st["w_next"].float()
    if not case["after"]:
        got = dict(y=(x * _rms(x) * wn).to(dt))
        if case["train"]:
            d, dw = _norm_back(x, wn, st["dy"].float())
            got.update(d_x=(st["dx"].float() + d).to(dt), d_w=dw.sum(0))
        return got
    h = st["h"].float()
    n = h * _rms(h) * st["w_post"].float() if case["post"] else h
    gate = st["gate"].float() if case["gate"] != "none" else 1.0
    new = x + st["scale"] * gate * n
    got = dict(x=new.to(dt), y=(new * _rms(new) * wn).to(dt))
    if not case["train"]:
        return got
    d, dw = _norm_back(got["x"].float(), wn, st["dy"].float())
    t = st["dx"].float() + d
    dn = st["scale"] * gate * t
    got.update(d_x=t.to(dt), d_w_next=dw.sum(0))
    if case["post"]:
        dh, dw = _norm_back(h, st["w_post"].float(), dn)
        got.update(d_h=dh.to(dt), d_w_post=dw.sum(0))
    else:
        got["d_h"] = dn.to(dt)
    if case["gate"] != "none":
        dg = st["scale"] * t * n
        got["d_gate"] = {"row": lambda: dg.sum(1, keepdim=True), "column": lambda: dg.sum(0), "full": lambda: dg.to(dt)}[case["gate"]]()
    return got


def _newton_schulz(u):
    a, b, c = COEF
    x = u / (u.square().sum((1, 2), keepdim=True).sqrt() + TINY)
    wide = x.shape[1] <= x.shape[2]
    for _ in range(STEPS):   # the iteration itself
        p = torch.bmm(x, x.transpose(1, 2)) if wide else torch.bmm(x.transpose(1, 2), x)
        q = b * p + c * torch.bmm(p, p)
        x = a * x + (torch.bmm(q, x) if wide else torch.bmm(x, q))
    return x


def _plain_ortho(st):
    g = st["g"].float()
    if not st["case"]["step"]:
        return dict(o=_newton_schulz(g).to(torch.bfloat16))
    m = MOMENTUM * st["m"] + g
    o = _newton_schulz(g + MOMENTUM * m)
    return dict(w=((1 - DECAY) * st["w"].float() - LR * o).to(st["w"].dtype), m=m)


def run(st):
    case = st["case"]
    if own:
        return _own(st)
    return {"ffn": _plain_ffn, "norm": _plain_norm, "ortho": _plain_ortho}[case["op"]](st)


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    import mixture_experts_expert_histogram_amd as moe
    case = st["case"]
    if case["op"] == "ffn":
        kw = dict(act=case["act"], layout=case["layout"], gate=st["gate"])
        out, saved, _ = moe.ffn_fwd(st["x"], st["gu"], st["dn"], add=st["add"], save=case["train"], **kw)
        if not case["train"]:
            return dict(out=out)
        dx, dgate, dgu, ddn, _ = moe.ffn_bwd(st["x"], st["gu"], st["dn"], st["dout"], saved=saved, **kw)
        got = dict(out=out, d_x=dx, d_gu=dgu, d_dn=ddn)
        if case["gated"]:
            got["d_gate"] = dgate
        return got
    if case["op"] == "norm" and not case["after"]:
        got = dict(y=moe.norm_fwd(st["x"], st["w_next"], eps=EPS))
        if case["train"]:
            got["d_x"], got["d_w"], _ = moe.norm_bwd(st["x"], st["w_next"], st["dy"], d_add=st["dx"], eps=EPS)
        return got
    if case["op"] == "norm":
        kw = dict(w_post=st["w_post"], gate=st["gate"], scale=st["scale"], w_next=st["w_next"], eps=EPS)
        x, y = moe.residual_fwd(st["x"], st["h"], **kw)
        got = dict(x=x, y=y)
        if case["train"]:
            d = moe.residual_bwd(x, st["h"], st["dx"], st["dy"], **kw)
            got.update(d_x=d.d_x, d_h=d.d_h, d_w_next=d.d_w_next)
            if case["post"]:
                got["d_w_post"] = d.d_w_post
            if case["gate"] != "none":
                got["d_gate"] = d.d_gate
        return got
    if not case["step"]:
        o, _ = moe.orthogonalize(st["g"], steps=STEPS, coef=COEF, eps=TINY)
        return dict(o=o)
    w, m, _ = moe.muon_step(st["w"], st["g"], st["m"], lr=LR, momentum=MOMENTUM, nesterov=True, decay=DECAY, steps=STEPS,
                            coef=COEF, eps=TINY, out=(torch.empty_like(st["w"]), torch.empty_like(st["m"])))
    return dict(w=w, m=m)


# ------------------------------------------------------------------ floors
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "ffn":
        T, H, I = case["T"], case["H"], case["I"]
        rows = T * H * size * (3 if case["gated"] else 2) + (4 * T if case["gated"] else 0)
        if not case["train"]:
            return dict(bytes=3 * H * I * size + rows, flops=6.0 * T * H * I)
        # forward: inputs, weights and out; backward: d_out read, d_x and the weight gradients written
        return dict(bytes=6 * H * I * size + rows + 2 * T * H * size, flops=18.0 * T * H * I)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        fwd, bwd = (2, 4) if not case["after"] else (4, 6)   # arrays [T,H] read and written
        full = case["gate"] == "full"
        n = fwd + full + (bwd + 2 * full if case["train"] else 0)
        return dict(bytes=n * T * H * size + 4 * H * size, flops=0)
    E, M, N = case["E"], case["M"], case["N"]
    s, l = min(M, N), max(M, N)
    # the two symmetric products need one triangle each
    flops = STEPS * (s * s * l + s * s * s + 2.0 * s * s * l) * E
    per = size + 2 + (2 + 8 if case["step"] else 0)
    return dict(bytes=E * M * N * per, flops=flops)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in st.items()}
    return {"ffn": _exact_ffn, "norm": _exact_norm, "ortho": _exact_ortho}[case["op"]](case, d, st)


def _exact_ffn(case, d, st):
    x, wd = d["x"], d["dn"]
    even = case["layout"] == "interleaved"
    wg, wu = (d["gu"][::2], d["gu"][1::2]) if even else d["gu"].chunk(2)
    g, u = x @ wg.T, x @ wu.T
    if case["act"] == "swiglu":
        s = 1 / (1 + torch.exp(-g))
        f, slope, v, inside = g * s, s + g * s * (1 - s), u, 1.0
    else:
        m = torch.minimum(g, torch.full_like(g, CLAMP))
        s = 1 / (1 + torch.exp(-ALPHA * m))
        f, slope = m * s, (s + ALPHA * m * s * (1 - s)) * (g <= CLAMP)
        v, inside = torch.clamp(u, -CLAMP, CLAMP) + 1, (u.abs() <= CLAMP).double()
    a = f * v
    p = 1 / (1 + torch.exp(-d["gate"])) if case["gated"] else torch.ones(len(x), dtype=x.dtype, device=x.device)
    out = p[:, None] * (a @ wd.T)
    if case["gated"]:
        out = out + d["add"]
    if not case["train"]:
        return dict(out=out)
    dy = p[:, None] * d["dout"]
    da = dy @ wd
    dg, du = da * v * slope, da * f * inside
    d_gu = torch.empty_like(d["gu"])
    rows = (slice(0, None, 2), slice(1, None, 2)) if even else (slice(0, case["I"]), slice(case["I"], None))
    d_gu[rows[0]], d_gu[rows[1]] = dg.T @ x, du.T @ x
    got = dict(out=out, d_x=dg @ wg + du @ wu, d_gu=d_gu, d_dn=dy.T @ a)
    if case["gated"]:
        got["d_gate"] = (1 - p) * (da * a).sum(1)
    return got


def _exact_rms(x, w):
    return w * x / torch.sqrt(x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS)


def _exact_norm(case, d, st):
    need = case["train"]
    x, wn = d["x"].requires_grad_(need), d["w_next"].requires_grad_(need)
    if not case["after"]:
        y = _exact_rms(x, wn)
        got = dict(y=y.detach())
        if need:
            dx, dw = torch.autograd.grad(y, (x, wn), d["dy"])
            got.update(d_x=dx + d["dx"], d_w=dw)
        return got
    leaves = {"d_h": d["h"].requires_grad_(need)}
    if case["post"]:
        leaves["d_w_post"] = d["w_post"].requires_grad_(need)
    if case["gate"] != "none":
        leaves["d_gate"] = d["gate"].requires_grad_(need)
    n = _exact_rms(d["h"], d["w_post"]) if case["post"] else d["h"]
    new = x + st["scale"] * (n if case["gate"] == "none" else d["gate"] * n)
    got = dict(x=new.detach(), y=_exact_rms(new, wn).detach())
    if need:
        # the backward pass takes the residual stream as the forward pass stored it
        held = new.detach().to(st["x"].dtype).double().requires_grad_()
        dnew, dw = torch.autograd.grad(_exact_rms(held, wn), (held, wn), d["dy"])
        t = dnew + d["dx"]
        got.update(d_x=t, d_w_next=dw)
        got.update(zip(leaves, torch.autograd.grad(new, list(leaves.values()), t)))
    return got


def _exact_ortho(case, d, st):
    a, b, c = COEF
    g = d["g"]
    if case["step"]:
        m = MOMENTUM * d["m"] + g
        g = g + MOMENTUM * m
    x = g / (torch.linalg.vector_norm(g, dim=(1, 2), keepdim=True) + TINY)
    if case["M"] > case["N"]:
        x = x.mT.contiguous()
    for _ in range(STEPS):
        p = x @ x.mT.contiguous()
        px = p @ x
        x = a * x + b * px + c * (p @ px)
    if case["M"] > case["N"]:
        x = x.mT
    return dict(w=(1 - DECAY) * d["w"] - LR * x, m=m) if case["step"] else dict(o=x)
