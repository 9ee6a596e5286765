"""Routing of up to 8192 slots by one workgroup, and of more by three passes: every output and the tables in the
workspace against the oracle's grouping, at the sizes where the passes and rounds change."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_histogram_amd as moe

pytestmark = pytest.mark.gpu

TILE_ROWS = (32, 64, 128, 256, 192)   # of the tables over every expert


def words(ws, at, n):
    return ws[at:at + 4 * n].view(torch.int32).cpu().numpy(), (at + 4 * n + 255) // 256 * 256


def check(ids, E):
    T, K = ids.shape
    f = ids.reshape(-1).astype(np.int64)
    key = np.where((f >= 0) & (f < E), f, E)
    order = np.argsort(key, kind="stable")
    count = np.bincount(key, minlength=E + 1)[:E]
    offset = np.concatenate(([0], np.cumsum(count)))
    inv = np.empty_like(f)
    inv[order] = np.arange(f.size)
    inv[key == E] = -1
    desc = moe.make_desc(T, 8, 8, E, K)
    ws = torch.full((moe.route_workspace_size(desc),), 0xFF, dtype=torch.uint8, device="cuda")
    counts, offsets, slots, pos, _ = moe.route(torch.from_numpy(ids).cuda(), E, ws=ws)
    torch.cuda.synchronize()
    assert np.array_equal(counts.cpu().numpy(), count)
    assert np.array_equal(offsets.cpu().numpy(), offset)
    assert np.array_equal(slots.cpu().numpy(), order)
    assert np.array_equal(pos.cpu().numpy(), inv)
    status, at = words(ws, 0, 4)
    assert status[0] == (key == E).sum()
    c, at = words(ws, at, E)
    o, at = words(ws, at, E + 1)
    assert np.array_equal(c, count) and np.array_equal(o, offset)
    tables, at = words(ws, at, 8 * (E + 1))
    tables = tables.reshape(8, E + 1)
    for j, rows in enumerate(TILE_ROWS):
        assert np.array_equal(tables[j], np.concatenate(([0], np.cumsum(-(-count // rows))))), rows
    by_count, at = words(ws, at, E)
    assert np.array_equal(by_count, np.argsort(-count, kind="stable"))


@pytest.mark.parametrize("S", [1, 63, 64, 65, 1000, 1023, 1024, 1025, 2047, 2048, 2049, 3333, 4095, 4096, 4097, 8191, 8192, 8193])
@pytest.mark.parametrize("E", [1, 3, 64, 127, 1024])
def test_sizes(S, E):
    rng = np.random.default_rng(S * 1031 + E)
    check(rng.integers(0, E, size=(S, 1)).astype(np.int32), E)


@pytest.mark.parametrize("T,K,E", [(1, 8, 8), (100, 8, 128), (512, 4, 128), (64, 64, 1000), (1, 64, 2), (683, 6, 33)])
def test_skewed_and_bad_ids(T, K, E):
    rng = np.random.default_rng(T + K + E)
    ids = np.minimum(rng.geometric(0.05, size=(T, K)) - 1, E - 1).astype(np.int32)
    check(ids, E)
    bad = rng.random((T, K)) < 0.1
    ids[bad] = rng.choice(np.array([-1, E, E + 5, -2 ** 31, 2 ** 31 - 1], dtype=np.int64), size=bad.sum()).astype(np.int32)
    check(ids, E)
    check(np.full((T, K), -1, dtype=np.int32), E)
    check(np.full((T, K), E - 1, dtype=np.int32), E)


def test_replays_and_ids_that_change():
    """A captured routing, replayed on other ids between eager calls."""
    E, T, K = 40, 300, 4
    rng = np.random.default_rng(7)
    ids = torch.from_numpy(rng.integers(0, E, size=(T, K)).astype(np.int32)).cuda()
    moe.route(ids, E)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = moe.route(ids, E)
    for _ in range(4):
        ids.copy_(torch.from_numpy(rng.integers(0, E, size=(T, K)).astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        want = moe.route(ids, E)
        torch.cuda.synchronize()
        for a, b in zip(got[:4], want[:4]):
            assert torch.equal(a, b)
