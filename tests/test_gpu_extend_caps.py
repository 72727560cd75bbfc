"""What decides how a capped score is computed: that score, and nothing else.

Bitwise where inputs that a row does not see change; against float64 for caps
far above the scores, where the capped score must keep fp32's accuracy relative
to itself: the bound is that of an uncapped call (extend_helpers), whose 16 spare
roundings a score also cover the cap's five and its fit (4.3e-8 of the score).
"""
import pytest
import torch

from tests.extend_helpers import DT, Batch, slopes

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", 64), ("bf16", 128), ("f16", 64), ("f16", 256), ("bf16", 256)]
LARGE = {"bf16": 1e6, "f16": 1e3, "f32": 1e6}


def leave_in_shared_memory(dtype, D, value):
    """A call on every SM whose outputs, staged where queries lie, are `value`."""
    b = Batch([(300, 300)] * 40, dtype, H=4, Hkv=2, D=D, seed=1)
    b.v.fill_(value)
    b.run(partition_tokens=-1)


@pytest.mark.parametrize("dtype,D", SHAPES)
@pytest.mark.parametrize("form", ["cap", "cap_alibi", "cap_window", "tree"])
def test_capped_results_do_not_depend_on_what_ran_before(dtype, D, form):
    lens = [(1, 400), (1, 70), (3, 200), (1, 1), (5, 129)] * 8
    b = Batch(lens, dtype, H=4, Hkv=2, D=D, seed=D)
    kw = dict(softcap=50.0, out_dtype=torch.float32, partition_tokens=-1)
    if "alibi" in form:
        kw["alibi_slopes"] = slopes(4)
    if "window" in form:
        kw["window"] = 40
    if form == "tree":
        kw["mask"] = b.tree_masks()
    leave_in_shared_memory(dtype, D, 0.0)
    first = b.run(**kw)
    for value in (LARGE[dtype], 0.0, -LARGE[dtype], LARGE[dtype]):
        leave_in_shared_memory(dtype, D, value)
        assert torch.equal(b.run(**kw), first), value


@pytest.mark.parametrize("dtype,D", SHAPES + [("f32", 128)])
def test_what_a_row_does_not_see_does_not_change_its_capped_scores(dtype, D):
    """Large finite values, infinities and NaN behind a context, in unused blocks,
    before every window, and in nodes that no mask holds."""
    lens = [(1, 5), (20, 100), (33, 161), (1, 300)]
    b = Batch(lens, dtype, H=4, Hkv=2, D=D, seed=11)
    kw = dict(softcap=50.0, out_dtype=torch.float32, partition_tokens=-1)
    mask = b.tree_masks()
    mask &= ~(1 << 7)  # node 7 is seen by none
    runs = [dict(), dict(window=40), dict(mask=mask), dict(alibi_slopes=slopes(4))]
    used = torch.zeros(b.NB, b.BS, dtype=torch.bool)
    for s, (n, c) in enumerate(lens):
        for j in range(c):
            used[int(b.tables[s, j // b.BS]), j % b.BS] = True
    dead = (~used).cuda()[:, None, :, None].expand_as(b.k)
    k0, v0 = b.k.clone(), b.v.clone()
    b.k[dead], b.v[dead] = 0, 0
    want = [b.run(**kw, **r) for r in runs]
    for value in (LARGE[dtype], float("inf"), float("nan")):
        b.k[dead], b.v[dead] = value, 1.0
        for r, w in zip(runs, want):
            assert torch.equal(b.run(**kw, **r), w), (value, r)
        for s, (n, c) in enumerate(lens):  # text that has left every window
            for j in range(max(0, c - n - 40 + 1)):
                b.k[int(b.tables[s, j // b.BS]), :, j % b.BS] = value
        assert torch.equal(b.run(**kw, window=40), want[1]), value
        b.k.copy_(k0), b.v.copy_(v0)
        b.k[dead], b.v[dead] = 0, 0
        for s, (n, c) in enumerate(lens):
            if n > 7:
                j = c - n + 7
                b.k[int(b.tables[s, j // b.BS]), :, j % b.BS] = value
        assert torch.equal(b.run(**kw, mask=mask), want[2]), value
        b.k.copy_(k0), b.v.copy_(v0)


@pytest.mark.parametrize("dtype,D", SHAPES + [("f32", 64)])
def test_other_queries_do_not_change_a_rows_capped_scores(dtype, D):
    b = Batch([(40, 300), (7, 7)], dtype, H=4, Hkv=2, D=D, seed=12)
    kw = dict(softcap=50.0, out_dtype=torch.float32, partition_tokens=-1)
    want = b.run(**kw)
    for value in (LARGE[dtype], float("inf"), float("nan")):
        b.q[3], b.q[20, 1], b.q[42, 2] = value, -value, value
        rest = torch.ones(b.T, 4, dtype=torch.bool, device="cuda")
        rest[3] = rest[20, 1] = rest[42, 2] = False
        assert torch.equal(b.run(**kw)[rest], want[rest]), value


@pytest.mark.parametrize("dtype,D", SHAPES + [("f32", 64)])
@pytest.mark.parametrize("cap", [1e3, 1e4, 1e5, 1e6, 1e9, 1e20, 1e35])
@pytest.mark.parametrize("one_large", [False, True])
def test_caps_far_above_the_scores(dtype, D, cap, one_large):
    """Few rows, so that most of a tile's are unused; with `one_large`, also a row
    whose scores pass 0.3 of the cap."""
    b = Batch([(1, 400), (2, 70), (5, 5)], dtype, H=4, Hkv=2, D=D, seed=13)
    rest = torch.ones(b.T, 4, dtype=torch.bool, device="cuda")
    if one_large:
        b.q[5, 2] *= min(8 * cap, 3e4 if dtype == "f16" else 1e15)
        rest[5, 2] = False
    for kw in (dict(), dict(alibi_slopes=slopes(4))):
        leave_in_shared_memory(dtype, D, LARGE[dtype]) if dtype != "f32" else None
        out = b.run(softcap=cap, out_dtype=torch.float32, **kw)
        rows, ref, _ = b.reference(softcap=cap, out_dtype=torch.float32, **kw)
        _, _, bound = b.reference(out_dtype=torch.float32, **kw)  # without the cap's own term
        off = (out[rows].double() - ref).abs()
        assert bool((off <= bound)[rest].all()), float((off / bound)[rest].max())


@pytest.mark.parametrize("dtype,D", SHAPES)
def test_scores_around_the_change_of_forms(dtype, D):
    """A tile whose scores lie on both sides of 0.3 of the cap, and one whose all
    lie below: the same scores give the same bits."""
    b = Batch([(40, 64)], dtype, H=2, Hkv=1, D=D, seed=14)
    kw = dict(softcap=1.0, out_dtype=torch.float32, partition_tokens=-1)
    b.q *= 0.02
    want = b.run(**kw)
    b.q[10:20] *= 60
    out = b.run(**kw)
    assert torch.equal(out[:10], want[:10]) and torch.equal(out[20:], want[20:])
    b.check(b.run(softcap=1.0), softcap=1.0)
    assert DT[dtype] == b.q.dtype
