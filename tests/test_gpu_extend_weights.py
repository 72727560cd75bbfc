"""Accuracy of the softmax weights of 16-bit pools: a lone key's value comes out
bit by bit, rounding is counted once, and small weights keep their bits."""
import math

import pytest
import torch

from tests.extend_helpers import HALF, Batch, slopes

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f16", 64), ("f16", 128), ("f16", 256)]


def values_of(b, s, j):
    """V [H][D] that query heads of sequence s have at position j."""
    return b.v[int(b.tables[s, j // b.BS]), :, j % b.BS].repeat_interleave(b.H // b.Hkv, 0)


@pytest.mark.parametrize("dtype,D", SHAPES)
@pytest.mark.parametrize("spread", [0.1, 1.0, 30.0])
@pytest.mark.parametrize("form", ["plain", "cap", "alibi"])
def test_a_token_that_sees_one_key_returns_its_value(dtype, D, spread, form):
    """The weight is 2^(a rounding of the score), off by |score| 2^-24 at most, and
    so is the sum: far less than half a step of the value."""
    b = Batch([(1, 1), (40, 40), (1, 1), (5, 300), (70, 200)], dtype, H=8, Hkv=2, D=D, seed=D, spread=spread)
    kw = {} if form == "plain" else dict(softcap=20.0) if form == "cap" else dict(alibi_slopes=slopes(8))
    first = b.run(**kw)
    for s in range(3):
        assert torch.equal(first[b.starts[s]], values_of(b, s, 0))
    for pt in (-1, 32):
        out = b.run(window=1, partition_tokens=pt, **kw)
        for s, (n, c) in enumerate(b.lens):
            for t in range(n):
                assert torch.equal(out[int(b.starts[s]) + t], values_of(b, s, c - n + t)), (s, t)
    if form != "alibi":  # nodes that see themselves only, with no text before them
        b = Batch([(40, 40), (9, 9)], dtype, H=8, Hkv=2, D=D, seed=D + 1, spread=spread)
        mask = torch.zeros(b.T, 2, dtype=torch.int32)
        for s, (n, _) in enumerate(b.lens):
            for i in range(n):
                bit = 1 << i % 32
                mask[int(b.starts[s]) + i, i // 32] = bit - (bit >> 31 << 32)
        out = b.run(mask.cuda(), **kw)
        for s, (n, _) in enumerate(b.lens):
            for i in range(n):
                assert torch.equal(out[int(b.starts[s]) + i], values_of(b, s, i))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_lone_key_in_tall_tiles(dtype):
    b = Batch([(300, 300), (40, 4500)], dtype, H=4, Hkv=2, D=128, seed=3).widen(5000)
    out = b.run(partition_tokens=-1)
    assert torch.equal(out[0], values_of(b, 0, 0))


@pytest.mark.parametrize("dtype,D", SHAPES)
@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_weights_are_rounded_once(dtype, D, out_dtype):
    """The bound with the weights' rounding in the numerator alone (the sum takes
    them as they are): extend_helpers' bound less its second count."""
    b = Batch([(1, 1), (2, 2), (3, 3), (16, 16), (1, 300), (37, 100), (64, 640)], dtype, H=8, Hkv=2, D=D, seed=D + 2)
    for kw in (dict(), dict(window=3), dict(mask=b.tree_masks())):
        out = b.run(out_dtype=out_dtype, **kw)
        rows, ref, bound = b.reference(out_dtype=out.dtype, **kw)
        half = HALF[b.dt]
        eps_p = half if out_dtype is None else half * half
        bound = bound - eps_p * ref.abs() * (1 + HALF[out.dtype])
        off = (out[rows].double() - ref).abs()
        assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("score", [-11.796875, -12.9921875, -13.4921875])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_fp16_weights_keep_their_bits(out_dtype, score, first, D):
    """One key of score 0 and value 0, and 2000 of weight e^score (2^-17 to 2^-19.5)
    and value 1: the result is made of the small weights alone.  They are normal
    fp16 numbers where the reference lies 2^7 below the largest score, so that their
    rounding is relative: half a step of 2^-11 (as two parts: of 2^-22, but no finer
    than 2^-25 of 2^7)."""
    n = 2000
    b = Batch([(1, n + 1)], "f16", H=1, Hkv=1, D=D, BS=256, seed=1)
    b.scale = 1.0
    b.q.zero_()
    b.q[..., 0] = 1.0
    b.k.zero_()
    b.k[..., 0] = score
    b.v.fill_(1.0)
    at = n if first else 0  # tiles are taken from the nearest keys on
    blk = int(b.tables[0, at // 256])
    b.k[blk, :, at % 256, 0] = 0.0
    b.v[blk, :, at % 256] = 0.0
    w = math.exp(score)
    ref = n * w / (1 + n * w)
    out = b.run(out_dtype=out_dtype, partition_tokens=-1).double()
    eps_p = 2.0 ** -11 if out_dtype == torch.float16 else 2.0 ** -22 + 2.0 ** -32 / w
    # the score as a power of 2: three roundings of 17 to 19.5 at 2^-24 each, ex2 2 ulp
    delta = 3 * 19.5 * 2.0 ** -24 + 2.0 ** -22
    bound = ref * (eps_p + 2 * delta + 2 * n * 2.0 ** -23)
    bound += HALF[out_dtype] * (ref + bound)
    assert float((out - ref).abs().max()) <= bound, float((out - ref).abs().max()) / bound


@pytest.mark.parametrize("D", [64, 128, 256])
def test_fp16_scores_that_grow_along_and_against_the_context(D):
    """The reference moves at every tile, and weights reach 2^15 before it does."""
    for order in (1, -1):
        b = Batch([(20, 900), (150, 600)], "f16", H=4, Hkv=2, D=D, seed=13)
        b.q[:] = b.q.abs()
        for s, (n, c) in enumerate(b.lens):
            for j in range(c):
                blk = int(b.tables[s, j // 16])
                x = j / c if order > 0 else 1 - j / c
                b.k[blk, :, j % 16] = b.k[blk, :, j % 16].abs() * (0.2 + 4 * x)
        for pt in (-1, 128):
            b.check(b.run(partition_tokens=pt))
            b.check(b.run(partition_tokens=pt, out_dtype=torch.float32))
            b.check(b.run(partition_tokens=pt, softcap=30.0), softcap=30.0)
    b = Batch([(150, 600)], "f16", H=4, Hkv=2, D=128, seed=14, spread=4.0).widen(5000)
    b.max_new = 300
    b.check(b.run())
