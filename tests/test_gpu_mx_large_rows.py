"""Rows to 4 bits and back where the largest grid (2^20 workgroups of 2^13 elements) goes round, ending inside a
workgroup's share: equal to the same rows in calls that do not go round, and the buffers left whole behind the last row."""
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_grid_goes_round(dtype):
    cols = 2080
    rows, pad = 2 ** 33 // cols + 34, 3
    assert 33 * cols < rows * cols - 2 ** 33 and rows * cols % 2 ** 13
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(1)
    parts = [slice(r, min(r + 500000, rows)) for r in range(0, rows, 500000)]
    w = torch.empty((rows, cols), dtype=tdt, device="cuda")
    for p in parts:
        w[p].normal_(generator=gen)
    w[-1, -32:] = 3.0
    codes = torch.full((rows + pad, cols // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + pad, cols // 32), 0xEE, dtype=torch.uint8, device="cuda")
    moe.mx_quantize(w, out=(codes[:rows], scales[:rows]))
    back = torch.full((rows + pad, cols), 7.0, dtype=tdt, device="cuda")
    moe.mx_dequantize(codes[:rows], scales[:rows], dtype=dtype, out=back[:rows])
    for p in parts:
        c, s = moe.mx_quantize(w[p])
        assert torch.equal(codes[p], c) and torch.equal(scales[p], s)
        assert torch.equal(back[p], moe.mx_dequantize(c, s, dtype=dtype))
    assert torch.all(back[rows - 1, -32:] == 3)
    assert torch.all(codes[rows:] == 0xEE) and torch.all(scales[rows:] == 0xEE) and torch.all(back[rows:] == 7)
    del w, codes, scales, back
    torch.cuda.empty_cache()
