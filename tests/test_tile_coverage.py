"""The shapes of the GPU tests run every instance of every dense product (no GPU is touched): a table of tile costs that
changes must not empty them unseen."""
import math
import random

from tests._tiles import FFN_SHAPES, FFN_VARIANTS, NAMES, STACKS, ffn_instances, ortho_instances

SQUARE = [n for n in NAMES if len(set(n.split("x"))) == 1]
FFN = ({("gate_up", n, v) for n in NAMES for v in ("swiglu", "clamped", "swiglu saved", "clamped saved", "recomputed")}
       | {(k, n, "") for n in NAMES for k in ("down", "gate_up_dgrad")} | {("down_dgrad", n, v) for n in NAMES for v in ("swiglu", "clamped")}
       | {("wgrad", n, v) for n in NAMES for v in ("bf16", "fp32")})
ORTHO = ({("gram", n, f) for n in SQUARE for f in ("wide", "tall")} | {("quad", n, "") for n in SQUARE}
         | {("update", n, f"{f} to {o}") for n in NAMES for f in ("wide", "tall") for o in ("X", "bf16", "fp32")})


def test_feed_forward_block():
    ran = set()
    for s in FFN_SHAPES:
        for act, _, grad in FFN_VARIANTS:
            ran |= ffn_instances(*s, act, grad == "fp32")
    assert ran == FFN


def test_orthogonalisation():
    assert set().union(*(ortho_instances(*s, out=("bf16", "fp32")) for s in STACKS)) == ORTHO


def test_nothing_else_can_run():
    rng = random.Random(0)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    for _ in range(3000):
        assert ffn_instances(log(17, 20000), 8 * log(1, 1100), 8 * log(1, 1100), "swiglu") <= FFN
        assert ortho_instances(log(1, 64), 8 * log(1, 720), 8 * log(1, 720)) <= ORTHO


def test_large_training_calls_run_on_the_largest_tiles():
    """The sizes of long training calls and of large stacks, and the shapes that stand for them here, choose alike."""
    assert {x[:2] for x in ffn_instances(8192, 4096, 8192, "swiglu")} == {x[:2] for x in ffn_instances(8185, 4072, 8152, "swiglu")}
    assert {x[1] for x in ffn_instances(8192, 4096, 8192, "swiglu")} == {"256x256"}
    assert ortho_instances(16, 2880, 2880) == ortho_instances(16, 2856, 2872)
    assert ortho_instances(8, 5760, 2880) == ortho_instances(8, 5752, 2872)
