"""The choice of tiles of the dense products (csrc/dense_tiles.h) on the host: which instances of which kernels a call runs.

The table is read from the source; the arithmetic is float32, as there."""
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_expert_histogram_amd", "csrc",
                      "dense_tiles.h")
F = np.float32
MAX_TILES = 1 << 23


def table():
    body = re.search(r"kTiles\[\] = \{(.*?)\};", open(SOURCE).read(), re.S).group(1)
    rows = re.findall(r"\{(\d+), (\d+), (\d+), ([\d.]+)f, ([\d.]+)f, ([\d.]+)f\}", body)
    assert len(rows) == 6
    return [(int(m), int(n), int(c), F(s), F(f), F(e)) for m, n, c, s, f, e in rows]


KINDS = table()
NAMES = [f"{64 * k[0]}x{64 * k[1]}" for k in KINDS]


def up(a, b):
    return -(-a // b)


def tile_time(k, tiles, K):
    nk = F(up(K, 64))
    if tiles <= 256:
        return (nk * k[3] + k[5]) * (F(0.65) + F(0.35) * F(tiles) / F(256))
    return F(up(tiles, 256 * k[2])) * (nk * k[4] + k[5])


def tile_kind(M, N, K, batch=1, first=0):
    best, least = first, F(0)
    for i in range(first, len(KINDS)):
        k = KINDS[i]
        tiles = batch * up(M, 64 * k[0]) * up(N, 64 * k[1])
        t = tile_time(k, tiles, K)
        if i == first or (t < least and tiles <= MAX_TILES):
            best, least = i, t
    return NAMES[best]


def square_tile_kind(S, K, batch):
    best, least = None, F(0)
    for i, k in enumerate(KINDS):
        if k[0] != k[1]:
            continue
        side = up(S, 64 * k[0])
        tiles = batch * side * (side + 1) // 2
        t = tile_time(k, tiles, K)
        if best is None or (t < least and tiles <= MAX_TILES):
            best, least = i, t
    return NAMES[best]


def ffn_instances(T, H, I, act, grad_fp32=False, few=16):
    """(kernel, tile, variant) of a bf16 block's forward pass with and without saved values and its backward pass with and
    without them; the forward pass of up to `few` tokens without saved values makes no tiles."""
    up_ = tile_kind(T, 2 * I, H)
    got = {("gate_up", up_, act + " saved"), ("gate_up", up_, "recomputed"), ("down", tile_kind(T, H, I), ""),
           ("down_dgrad", tile_kind(T, I, H), act), ("gate_up_dgrad", tile_kind(T, H, 2 * I), "")}
    if T > few:
        got.add(("gate_up", up_, act))
    kind = "fp32" if grad_fp32 else "bf16"
    return got | {("wgrad", tile_kind(H, I, T), kind), ("wgrad", tile_kind(2 * I, H, T), kind)}


def ortho_instances(E, M, N, out=("bf16",), steps=5):
    """(kernel, tile, variant) of an orthogonalisation with results of the given types, or of a step of such weights."""
    S, L = min(M, N), max(M, N)
    form = "wide" if M <= N else "tall"
    tile = tile_kind(M, N, S, E, 3 if S < 64 else 0)
    got = {("gram", square_tile_kind(S, L, E), form), ("quad", square_tile_kind(S, S, E), "")}
    got |= {("update", tile, f"{form} to {o}") for o in out}
    return got | ({("update", tile, form + " to X")} if steps > 1 else set())


# Shapes, none of whole tiles, that between them run every kernel on every tile it can have, and large ones of many steps of k
FFN_SHAPES = [(213, 168, 160), (5560, 168, 176), (434, 200, 4144), (3710, 376, 160), (8203, 496, 496), (4652, 1952, 2920),
              (3037, 4120, 168), (2075, 1160, 4648), (8185, 4072, 8152)]
FFN_VARIANTS = [("swiglu", "concat", None), ("clamped", "interleaved", "fp32")]
STACKS = [(1, 8, 8), (45, 152, 136), (53, 200, 8), (56, 264, 280), (44, 144, 248), (55, 456, 408), (46, 296, 288), (58, 80, 72),
          (37, 72, 784), (43, 968, 72), (61, 408, 528), (56, 136, 776), (16, 2856, 2872), (8, 5752, 2872)]
