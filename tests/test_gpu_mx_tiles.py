"""The grouped products on 4-bit weights, per tile height and number of 128-k stages.

A tile of 32 positions (at most 16 slots an expert on average) loads the codes of 4 stages of a row together and goes round
its loop body once for 8 stages, a tile of 64 those of 2 and goes round once for 4; what is left runs behind a question a
stage.  The sizes below leave every remainder in both products, with and without rounds of the loop before it, and end
inside a stage as well as on one.  The experts' counts put one and two (32) and one to four (64) blocks of 16
positions in a tile, several tiles on an expert, and none."""
import numpy as np
import pytest

from tests._gpu import small_inputs
from tests.test_gpu_mx import mx_case

E = 10
COUNTS = {32: [0, 1, 16, 17, 32, 33, 40, 21, 0, 0], 64: [0, 1, 16, 33, 48, 49, 64, 65, 100, 24]}

pytestmark = pytest.mark.gpu


def stages(n):
    """A row length of n stages, short of them by 0 to 3 blocks."""
    return 128 * n - 32 * (n % 4)


def run(rows, H, I, act, layout):
    counts = COUNTS[rows]
    T = sum(counts)
    assert T > 128 and (T <= 16 * E) == (rows == 32)
    ids = np.random.default_rng(H + I).permutation(np.repeat(np.arange(E), counts)).astype(np.int32).reshape(T, 1)
    mx_case(small_inputs(T, H, I, E, 1, "bf16", act, layout, seed=H + I, ids=ids))


@pytest.mark.parametrize("rows", [32, 64])
@pytest.mark.parametrize("n", range(1, 9))
def test_remainders(n, rows):
    """1 to 8 stages in the gate_up product, 9 to 2 in the down product."""
    run(rows, stages(n), stages(10 - n), *(("clamped", "interleaved") if n % 2 else ("swiglu", "concat")))


@pytest.mark.parametrize("rows", [32, 64])
@pytest.mark.parametrize("n", [11, 14, 15])
def test_remainders_behind_a_round_of_the_loop(n, rows):
    run(rows, stages(n), stages(24 - n), "clamped", "concat")


@pytest.mark.parametrize("rows", [32, 64])
@pytest.mark.parametrize("H,I,act,layout", [(2880, 1440, "clamped", "interleaved"), (1440, 2880, "swiglu", "concat"),
                                            (2080, 544, "clamped", "concat")])
def test_long_rows_off_a_stage(H, I, act, layout, rows):
    """2880: 23 stages, the last of 64 k; 2080: 17, the last of 32."""
    run(rows, H, I, act, layout)
