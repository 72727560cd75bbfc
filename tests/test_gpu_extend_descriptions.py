"""Sequences described wrongly, in calls that split the context: rows come out
untouched or computed, never from parts that the call did not write."""
import pytest
import torch

from paged_kv_cache_249_gb300 import pagedkv
from tests.extend_helpers import Batch

pytestmark = pytest.mark.gpu

LENS = [(100, 600), (60, 600), (140, 600), (300, 600)]
T = 600
# (the first two name more rows than there are, so that items find no room)
WRONG = [[0, T, 0, T, T], [0, T, 0, T, 0], [0, T - 5, 3, T - 4, 1], [0, 40, 30, 150, T], [0, 40, 100, 150, T + 1],
         [-1, 40, 100, 150, T], [0, 40, 1 << 30, 150, T], [T, 150, 100, 40, 0], [40, T, 10, T, T],
         [-(1 << 31), 0, T, 0, (1 << 31) - 1]]


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f16", 256), ("f32", 64)])
@pytest.mark.parametrize("wrong", WRONG, ids=str)
@pytest.mark.parametrize("tree", [False, True])
def test_starts_out_of_order_or_range(dtype, D, wrong, tree):
    b = Batch(LENS, dtype, H=8, Hkv=2, D=D, seed=17)
    b.max_new = T
    mask = b.tree_masks(words=-(-T // 32)) if tree else None
    ws = b.workspace(32)
    good = b.run(mask, partition_tokens=32, workspace=ws)
    assert bool(torch.isfinite(good).all())
    b.starts.copy_(torch.tensor(wrong, dtype=torch.int64).to(torch.int32))
    ws.view(torch.float32).fill_(float("nan"))
    out = b.run(mask, partition_tokens=32, workspace=ws, out=torch.full_like(good, 7.0))
    torch.cuda.synchronize()
    assert pagedkv.get_device_error(b.pool) == pagedkv.FAULT_QUERY
    assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_sequence_that_is_too_long_leaves_the_others_computed(dtype):
    b = Batch(LENS, dtype, H=4, Hkv=2, D=64, seed=18)
    ws = b.workspace(32)
    good = b.run(partition_tokens=32, workspace=ws)
    b.max_new = 299  # the last sequence brings 300
    ws.view(torch.float32).fill_(float("nan"))
    out = b.run(partition_tokens=32, workspace=ws, out=torch.full_like(good, 7.0))
    torch.cuda.synchronize()
    assert pagedkv.get_device_error(b.pool) == pagedkv.FAULT_QUERY
    assert torch.equal(out[:300], good[:300]) and bool((out[300:] == 7.0).all())


def test_more_sequences_than_are_listed_at_once():
    """Beyond 512 sequences items are found by another rule."""
    lens = [(1 + s % 3, 40 + s % 50) for s in range(600)]
    b = Batch(lens, "bf16", H=4, Hkv=2, D=64, seed=19)
    ws = b.workspace(32)
    good = b.run(partition_tokens=32, workspace=ws)
    b.check(good)
    starts = b.starts.clone()
    for at, to in ((300, 0), (300, b.T), (1, b.T), (599, 0)):
        b.starts.copy_(starts)
        b.starts[at] = to
        ws.view(torch.float32).fill_(float("nan"))
        out = b.run(partition_tokens=32, workspace=ws, out=torch.full_like(good, 7.0))
        torch.cuda.synchronize()
        assert pagedkv.get_device_error(b.pool) == pagedkv.FAULT_QUERY
        assert bool(torch.isfinite(out).all())
