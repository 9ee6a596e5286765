"""Cases of the serving operators of the MoE layer, with their plain forms.

Three operators, all of the layer  out[t] = sum_k w[t,k] Wd[e] phi(Wgu[e] x_t),
e = ids[t,k]:

* "few":   the layer for a few tokens, bf16 or fp32 weights;
* "quant": weight rows to 4-bit microscaled floating point (E2M1 codes, one
           power-of-two E8M0 scale for 32 consecutive elements) and back;
* "mx":    the layer on weights held in that form, from one token to thousands.

Layer sizes are those of the repository's workloads (gpt-oss-shaped
H = I = 2880, E = 128, top-4; H = 4096, I = 2048, E = 256, top-8) and small
ragged ones.  `own` selects the framework's calls; otherwise the operators are
computed by elementary torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

CLAMP, ALPHA = 7.0, 1.702
BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _layer(name, op, T, H, I, E, K, act, layout, dtype="bf16", logits=False):
    return dict(name=name, op=op, T=T, H=H, I=I, E=E, K=K, act=act, layout=layout, dtype=dtype, logits=logits)


def listed():
    return [
        # one token through one gpt-oss-shaped layer, as each step of a single chat decodes (from router logits)
        _layer("few 1 token", "few", 1, 2880, 2880, 128, 4, "clamped", "interleaved", logits=True),
        # a small batch of chats decoding together: most experts hold one token
        _layer("few 16 tokens", "few", 16, 2880, 2880, 128, 4, "clamped", "interleaved"),
        # top-8 of 256 narrow experts, a larger decode batch: nearly every expert is read
        _layer("few 48 tokens top-8", "few", 48, 4096, 2048, 256, 8, "swiglu", "concat"),
        # a ragged fp32 layer at small size: latency, odd row counts
        _layer("few 5 tokens fp32 ragged", "few", 5, 1048, 712, 12, 3, "swiglu", "concat", dtype="fp32"),
        # a checkpoint's bf16 expert weights to 4 bits and back: 16 experts' gate_up rows
        dict(name="quant bf16 weights", op="quant", rows=16 * 5760, cols=2880, dtype="bf16"),
        # an odd number of short fp32 rows (one expert's matrix of a small layer)
        dict(name="quant fp32 odd rows", op="quant", rows=1337, cols=736, dtype="fp32"),
        # the single-token step on 4-bit weights (from router logits)
        _layer("mx 1 token", "mx", 1, 2880, 2880, 128, 4, "clamped", "interleaved", logits=True),
        # a decode batch on 4-bit weights
        _layer("mx 32 tokens", "mx", 32, 2880, 2880, 128, 4, "clamped", "interleaved"),
        # a short prompt, or a large decode batch: about 16 tokens an expert
        _layer("mx 512 tokens", "mx", 512, 2880, 2880, 128, 4, "clamped", "interleaved"),
        # prompts of the top-8 layer: about 64 tokens an expert
        _layer("mx 2048 tokens top-8", "mx", 2048, 4096, 2048, 256, 8, "swiglu", "concat"),
        # a prompt chunk, the repository's gpt-oss-shaped token count: about 128 tokens an expert
        _layer("mx 4096 tokens", "mx", 4096, 2880, 2880, 128, 4, "clamped", "interleaved"),
        # a ragged small layer, token count off every tile
        _layer("mx 77 tokens ragged", "mx", 77, 1056, 736, 10, 3, "clamped", "concat"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Sizes of the same three operators, over the ranges between the listed cases."""
    op = rng.choice(["few", "few", "quant", "mx", "mx", "mx"])
    if op == "quant":
        dtype = rng.choice(["bf16", "fp32"])
        cols = BLOCK * _log(rng, 1, 256)
        return dict(op=op, rows=_log(rng, 1, max(1, (64 << 20) // cols)), cols=cols, dtype=dtype)
    unit = 8 if op == "few" else BLOCK
    H, I = unit * _log(rng, 256 // unit, 4096 // unit), unit * _log(rng, 256 // unit, 2880 // unit)
    E = min(_log(rng, 4, 256), (128 * 2880 * 2880) // (H * I))
    K = min(rng.choice([1, 2, 4, 8]), E)
    dtype = "bf16" if op == "mx" else rng.choice(["bf16", "bf16", "fp32"])
    T = _log(rng, 1, 128) if op == "few" else max(1, min(_log(rng, 1, 4096), (4096 * 4 * 2880 * 2880) // (K * H * I)))
    c = _layer("", op, T, H, I, E, K, rng.choice(["swiglu", "clamped"]), rng.choice(["concat", "interleaved"]), dtype,
               logits=rng.random() < 0.4)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    """Weights as a program loads them once; hidden states N(0,1) after a norm; router logits N(0,1) with experts of
    uneven popularity."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "quant":
        # rows of different size, as the output channels of a trained matrix have
        w = torch.randn((case["rows"], case["cols"]), generator=g, device=dev, dtype=dt)
        w *= (0.02 * torch.exp(0.5 * torch.randn((case["rows"], 1), generator=g, device=dev))).to(dt)
        return dict(case=case, w=w)
    T, H, I, E, K = (case[n] for n in ("T", "H", "I", "E", "K"))
    st = dict(case=case)
    st["hidden"] = torch.randn((T, H), generator=g, device=dev, dtype=torch.float32).to(dt)
    lg = torch.randn((T, E), generator=g, device=dev) + 0.3 * torch.randn((1, E), generator=g, device=dev)
    if case["logits"]:
        st["logits"] = lg
    else:
        top = torch.topk(lg, K, dim=1)
        st["ids"] = top.indices.to(torch.int32)
        st["weights"] = torch.softmax(top.values, dim=1)
    for name, rows, cols in (("gu", 2 * I, H), ("dn", H, I)):
        if case["op"] == "few":
            st[name] = torch.randn((E, rows, cols), generator=g, device=dev, dtype=dt).mul_(0.02)
        else:
            codes = torch.empty((E, rows, cols // 2), dtype=torch.uint8, device=dev)
            scales = torch.empty((E, rows, cols // BLOCK), dtype=torch.uint8, device=dev)
            n = max(1, (64 << 20) // (rows * cols))
            for e in range(0, E, n):
                w = torch.randn((min(n, E - e), rows, cols), generator=g, device=dev).mul_(0.02)
                code, shared = _codes(w)
                codes[e:e + n] = code[..., 0::2] | (code[..., 1::2] << 4)
                scales[e:e + n] = (shared + 127).to(torch.uint8)
            st[name] = (codes, scales)
    return st


# ------------------------------------------------------------------ the plain forms
def _two_to(n):
    """2^n in fp32 for whole n from -126 to 127, from the bits (a power function may be an ulp off)."""
    return ((n + 127) << 23).view(torch.float32)


def _codes(w):
    """E2M1 codes (uint8, one an element) and shared exponents (one for 32 elements) of finite rows: the shared exponent
    is floor(log2(max |w|)) - 2 (at least -127), the code the nearest of w / 2^shared, ties to the even code, magnitudes
    over 6 to 6."""
    x = w.float().reshape(w.shape[:-1] + (w.shape[-1] // BLOCK, BLOCK))
    amax = x.abs().amax(-1)
    shared = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127).to(torch.int32)
    m = x * _two_to(-shared)[..., None]
    s = torch.signbit(m)
    m = m.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    return (code + 8 * s.to(torch.uint8)).reshape(w.shape), shared


def _values(codes, shared):
    """What codes and shared exponents stand for, in fp32."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    x = table[codes.int()].reshape(shared.shape + (BLOCK,))
    return (0.5 * x * _two_to(shared + 1)[..., None]).reshape(codes.shape)   # 2^-127 itself is subnormal


def _weights(w, active):
    """Expert weights of the chosen experts, fp32."""
    if not isinstance(w, tuple):
        return w[active].float()
    codes, scales = w[0][active], w[1][active]
    pair = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pair = torch.stack((pair.repeat(16), pair.repeat_interleave(16)), dim=1)   # byte -> its low, then its high element
    x = pair[codes.int()].reshape(scales.shape + (BLOCK,))
    x *= 0.5 * _two_to(scales.int() - 126)[..., None]
    return x.reshape(codes.shape[:-1] + (codes.shape[-1] * 2,))


def _route(st):
    """(ids, weights) given or chosen: the K largest logits, equal ones by the lower id; their softmax."""
    case = st["case"]
    if not case["logits"]:
        return st["ids"].long(), st["weights"]
    top, ids = torch.sort(st["logits"], dim=1, descending=True, stable=True)
    top, ids = top[:, :case["K"]], ids[:, :case["K"]]
    z = torch.exp(top - top[:, :1])
    return ids, z / z.sum(1, keepdim=True)


def _glu(z, case):
    if case["layout"] == "interleaved":
        gate, up = z[..., 0::2], z[..., 1::2]
    else:
        gate, up = z[..., :case["I"]], z[..., case["I"]:]
    if case["act"] == "swiglu":
        return gate * torch.sigmoid(gate) * up
    gate, up = gate.clamp(max=CLAMP), up.clamp(-CLAMP, CLAMP)
    return (up + 1) * gate * torch.sigmoid(ALPHA * gate)


def _plain_layer(st):
    case = st["case"]
    T, H, K = case["T"], case["H"], case["K"]
    ids, w = _route(st)
    # the slots grouped by expert, each group padded to the largest one
    active, of, counts = torch.unique(ids.reshape(-1), return_inverse=True, return_counts=True)
    order = torch.argsort(of, stable=True)
    group = of[order]
    place = torch.arange(T * K, device=ids.device) - (torch.cumsum(counts, 0) - counts)[group]
    x = torch.zeros((active.numel(), int(counts.max()), H), device=ids.device)
    x[group, place] = st["hidden"].float()[order // K]
    z = torch.bmm(x, _weights(st["gu"], active).transpose(1, 2))
    y = torch.bmm(_glu(z, case), _weights(st["dn"], active).transpose(1, 2))
    slots = torch.empty((T * K, H), device=ids.device)
    slots[order] = y[group, place]
    out = (slots.reshape(T, K, H) * w[..., None]).sum(1).to(DTYPES[case["dtype"]])
    return _answer(case, out, ids.to(torch.int32), w)


def _answer(case, out, ids, w):
    return dict(out=out, ids=ids, weights=w) if case["logits"] else dict(out=out)


def run(st):
    case = st["case"]
    if own:
        import mixture_experts_expert_histogram_amd as moe
        if case["op"] == "quant":
            codes, scales = moe.mx_quantize(st["w"])
            return dict(values=moe.mx_dequantize(codes, scales, dtype=case["dtype"]))
        kw = dict(act=case["act"], layout=case["layout"])
        if case["logits"]:
            call = moe.fwd_few_logits if case["op"] == "few" else moe.mx_fwd_logits
            out, ids, w, _ = call(st["hidden"], st["logits"], case["K"], st["gu"], st["dn"], **kw)
            return _answer(case, out, ids, w)
        call = moe.fwd_few if case["op"] == "few" else moe.mx_fwd
        out, _ = call(st["hidden"], st["ids"], st["weights"], st["gu"], st["dn"], **kw)
        return _answer(case, out, None, None)
    if case["op"] == "quant":
        codes, shared = _codes(st["w"])
        return dict(values=_values(codes, shared).to(st["w"].dtype))
    return _plain_layer(st)


# ------------------------------------------------------------------ floors
def work(case):
    if case["op"] == "quant":
        n, size = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        held = n // 2 + n // BLOCK
        return dict(bytes=2 * n * size + 2 * held, flops=0)
    T, H, I, E, K = (case[n] for n in ("T", "H", "I", "E", "K"))
    size = 2 if case["dtype"] == "bf16" else 4
    per = 0.5 + 1 / BLOCK if case["op"] == "mx" else size
    active = E * (1 - (1 - K / E) ** T)   # experts that uniform routing reaches
    return dict(bytes=active * 3 * H * I * per + 2 * T * H * size + T * K * 8 + (T * E * 4 if case["logits"] else 0),
                flops=6.0 * T * K * H * I)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        return dict(values=_exact_quant(st["w"]))
    K = case["K"]
    x = st["hidden"].double()
    if case["logits"]:
        lg = st["logits"].double()
        ids = torch.argsort(lg, dim=1, descending=True, stable=True)[:, :K]
        w = torch.softmax(torch.gather(lg, 1, ids), dim=1)
    else:
        ids, w = st["ids"].long(), st["weights"].double()
    out = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=x.device)
    for e in torch.unique(ids).tolist():
        t, k = torch.nonzero(ids == e, as_tuple=True)
        z = x[t] @ _exact_expert(st["gu"], e).T
        even = case["layout"] == "interleaved"
        gate, up = (z[:, ::2], z[:, 1::2]) if even else z.chunk(2, dim=1)
        if case["act"] == "swiglu":
            a = gate / (1 + torch.exp(-gate)) * up
        else:
            gate, up = torch.clamp(gate, max=CLAMP), torch.clamp(up, -CLAMP, CLAMP)
            a = (up + 1) * gate / (1 + torch.exp(-ALPHA * gate))
        out.index_add_(0, t, (a @ _exact_expert(st["dn"], e).T) * w[t, k][:, None])
    return dict(out=out, ids=None, weights=w) if case["logits"] else dict(out=out)


def _exact_expert(w, e):
    if not isinstance(w, tuple):
        return w[e].double()
    byte = w[0][e].long()
    code = torch.stack((byte % 16, byte // 16), dim=-1).reshape(byte.shape[0], -1)
    sign, exponent, mantissa = 1 - 2 * (code // 8), (code // 2) % 4, (code % 2).double()
    v = torch.where(exponent > 0, (1 + mantissa / 2) * _exact_two_to(exponent - 1), mantissa / 2) * sign
    return v * _exact_two_to(w[1][e].long() - 127).repeat_interleave(BLOCK, dim=1)


def _exact_two_to(n):
    """2^n in 64 bits, from the bits."""
    return ((n + 1023) << 52).view(torch.float64)


def _exact_quant(w):
    """The nearest representable value of each element, block by block, in chunks of rows."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=w.device)
    parts = []
    for rows in w.split(max(1, (32 << 20) // w.shape[1])):
        x = rows.double().reshape(rows.shape[0], -1, BLOCK)
        top = x.abs().amax(-1, keepdim=True)
        step = torch.where(top > 0, ((top.view(torch.int64) >> 52) - 1023) - 2, -127)   # floor(log2(top)) - 2
        scale = _exact_two_to(step.clamp(-127, 127))
        m = (x / scale).abs()
        i = torch.searchsorted(grid, m.contiguous()).clamp(1, 7)      # grid[i - 1] < m <= grid[i], or m past the ends
        lo, hi = grid[i - 1], grid[i]
        up = (m - lo > hi - m) | ((m - lo == hi - m) & (i % 2 == 0))   # ties to the even code
        parts.append((torch.where(up, hi, lo) * torch.sign(x) * scale).reshape(rows.shape))
    return torch.cat(parts)
