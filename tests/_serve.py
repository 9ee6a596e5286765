"""Helpers of the serving-operator tests: a 64-bit reference of the layer with
an elementwise error bound, and the 4-bit format in 64 bits.

The bound (layer_bound) is first order and worst case.  Roundings, each at
most half a step: a = phi(g, u) to the activations' type (u = 2^-8 bf16, 2^-24
fp32), the output (the same u), and fp32 sums of n terms (n 2^-24 of the sum of
the terms' magnitudes, which covers any order).  The gate and up sums' errors
pass through phi's derivative; the logistic function's own error is taken as
2^-17 |a| (hardware exp2 and reciprocal at about 1 ulp each, an argument
rounded to 24 bits and at most 2^6 in size).  The factor 1.01 covers the
products of two such terms.
"""
import numpy as np

import oracle

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def layer_bound(X, ids, w, experts, act, layout, dtype, limit=7.0, alpha=1.702):
    """(out, bound) in fp64: the layer's output and the largest error of an
    implementation with the roundings above.  Slots with an id outside the
    experts are dropped.  experts: list of (w_gate_up, w_down)."""
    X = np.asarray(X, dtype=np.float64)
    T, H = X.shape
    out, err = np.zeros((T, H)), np.zeros((T, H))
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    K = ids.shape[1]
    for e, (gu, dn) in enumerate(experts):
        t, k = np.nonzero(ids == e)
        if t.size == 0:
            continue
        gu, dn = np.asarray(gu, dtype=np.float64), np.asarray(dn, dtype=np.float64)
        I = dn.shape[1]
        g, up = oracle.split_gate_up(X[t] @ gu.T, layout)
        eg, eu = oracle.split_gate_up(np.abs(X[t]) @ np.abs(gu).T * (H * 2.0 ** -24), layout)
        a = oracle.glu(g, up, act, limit, alpha)
        # phi' from the backward of a unit gradient; at the clamps both sides' slopes are at most the inner one's
        dg, du = oracle.glu_backward(g, up, np.ones_like(a), act, limit, alpha)
        if act == "clamped":   # a value within its error of a clamp may fall on either side
            dg2, du2 = oracle.glu_backward(np.minimum(g, limit), np.clip(up, -limit, limit), np.ones_like(a), act, limit, alpha)
            dg, du = np.maximum(np.abs(dg), np.abs(dg2)), np.maximum(np.abs(du), np.abs(du2))
        ea = np.abs(dg) * eg + np.abs(du) * eu + (u + 2.0 ** -17) * np.abs(a)
        wt = np.asarray(w, dtype=np.float64)[t, k][:, None]
        np.add.at(out, t, wt * (a @ dn.T))
        mag = np.abs(a) @ np.abs(dn).T
        np.add.at(err, t, np.abs(wt) * (ea @ np.abs(dn).T + (I + K + 1) * 2.0 ** -24 * mag))
    return out, 1.01 * (err + u * (np.abs(out) + err))


def check_layer(got, ref, bound, name=""):
    """Elementwise within the bound, and in the 2-norm within 2^-7 (bf16: two
    roundings of at most 2^-8 each, a's spread over the sum like the sum
    itself) of the reference."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape
    assert np.all(np.isfinite(got)), f"{name}: non-finite values"
    over = np.abs(got - ref) - bound
    assert np.max(over, initial=-1.0) <= 0, f"{name}: {np.max(over):.3e} past the bound at {np.unravel_index(np.argmax(over), over.shape)}"
    n = np.linalg.norm(ref)
    if n > 0:
        assert np.linalg.norm(got - ref) <= 2.0 ** -7 * n, f"{name}: relative error {np.linalg.norm(got - ref) / n:.3e}"


def quantize_ref(w):
    """(codes, scale bytes) one an element / block of 32, in fp64: the format's
    definition, by search over the eight magnitudes."""
    with np.errstate(invalid="ignore"):   # signalling NaNs
        x = np.asarray(w, dtype=np.float64).reshape(-1, 32)
    codes = np.zeros(x.shape, dtype=np.uint8)
    scales = np.zeros(len(x), dtype=np.uint8)
    for b, row in enumerate(x):
        if not np.all(np.isfinite(row)):
            scales[b] = 255
            continue
        top = np.max(np.abs(row))
        shared = -127 if top == 0 else max(int(np.frexp(top)[1]) - 1 - 2, -127)
        scales[b] = shared + 127
        m = np.abs(row) / 2.0 ** shared
        d = np.abs(m[:, None] - E2M1[None, :])
        near = d.min(axis=1)
        for i in range(32):
            best = np.nonzero(d[i] == near[i])[0]
            c = best[0] if len(best) == 1 else next(v for v in best if v % 2 == 0)
            codes[b, i] = c + (8 if np.signbit(row[i]) else 0)
    return codes, scales


def pack(codes):
    """[n, 32] codes -> [n, 16] bytes."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def values_ref(packed, scales):
    """fp64 values of packed codes [..., C/2] and scales [..., C/32]; blocks of scale 255 are NaN."""
    packed, scales = np.asarray(packed), np.asarray(scales)
    c = np.stack((packed & 15, packed >> 4), axis=-1).reshape(packed.shape[:-1] + (packed.shape[-1] * 2,))
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=-1)
