"""Values that are not finite: which results they reach and as what, and that a
call with a few of them takes no more than a few times as long."""
import math

import pytest
import torch

from tests.extend_helpers import Batch

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f16", 64), ("f16", 128), ("f16", 256)]
LENS = [(60, 150), (20, 20), (1, 100), (3, 70)]


def expected(b, mask=None, softcap=0.0, window=0, prefix_lens=None):
    """Rows in float64 from the keys that each row sees and no others, in whose
    sums infinities and NaN follow IEEE arithmetic."""
    G, dev = b.H // b.Hkv, b.q.device
    out = torch.zeros(b.q.shape, dtype=torch.float64, device=dev)
    starts = b.starts.tolist()
    for s, (n, ctx) in enumerate(b.lens):
        j = torch.arange(ctx, device=dev)
        blk = b.tables[s].long()[j // b.BS]
        k, v = (x[blk, :, j % b.BS].double().repeat_interleave(G, 1) for x in (b.k, b.v))
        p = (ctx - n + torch.arange(n, device=dev))[:, None]
        if mask is not None:
            m, bit = mask[starts[s]:starts[s + 1]].long(), torch.arange(n, device=dev)
            seen = torch.cat([torch.ones(n, ctx - n, dtype=torch.bool, device=dev),
                              (m[:, bit // 32] >> (bit % 32) & 1).bool()], 1)
        else:
            seen = j <= p
            if prefix_lens is not None:
                seen = seen | (j < prefix_lens[s])
            if window:
                seen = seen & (p - j < window)
        for t in range(n):
            at = seen[t].nonzero()[:, 0]
            if len(at) == 0:
                continue
            z = torch.einsum("hd,jhd->hj", b.q[starts[s] + t].double(), k[at]) * b.scale
            if softcap:
                z = softcap * torch.tanh(z / softcap)
            w = torch.softmax(z, -1)
            out[starts[s] + t] = (w.T[..., None] * v[at]).sum(0)
    return out


def sprinkle(b, seed, what):
    """Some keys of the sequences get values that are not finite, in some columns;
    returns what to put back."""
    g = torch.Generator().manual_seed(seed)
    for s, (n, ctx) in enumerate(b.lens):
        for _ in range(3):
            j = int(torch.randint(max(0, ctx - n - 5), ctx, (1,), generator=g))
            col = torch.randperm(b.D, generator=g)[:3].to(b.v.device)
            head = int(torch.randint(0, b.Hkv, (1,), generator=g))
            value = what[int(torch.randint(0, len(what), (1,), generator=g))]
            b.v[int(b.tables[s, j // b.BS]), head, j % b.BS, col] = value


def same_kind(out, want, clean, bound):
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.isinf(), want.isinf())
    inf = want.isinf()
    assert torch.equal(out.double()[inf], want[inf])
    ok = torch.isfinite(want)
    off = (out.double() - want).abs()
    assert bool((off <= bound)[ok].all()), float((off / bound)[ok].max())


@pytest.mark.parametrize("dtype,D", SHAPES)
@pytest.mark.parametrize("what", [(math.inf,), (math.nan,), (math.inf, -math.inf, math.nan)], ids=str)
@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_each_reaches_the_tokens_that_see_it_as_what_it_is(dtype, D, what, out_dtype):
    for seed in range(2):
        b = Batch(LENS, dtype, H=4, Hkv=2, D=D, seed=12 + seed)
        mask = b.tree_masks(3)
        prefix = torch.tensor([120, 7, 0, 69], dtype=torch.int32, device="cuda")
        forms = [dict(), dict(window=16), dict(mask=mask), dict(prefix_lens=prefix), dict(softcap=5.0)]
        # (bounds of the finite values; those put in are seen by no finite result)
        clean = [b.reference(out_dtype=out_dtype, **kw) for kw in forms]
        sprinkle(b, seed, what)
        for kw, (_, ref, bound) in zip(forms, clean):
            want = expected(b, **kw)
            for pt in (-1, 32):
                same_kind(b.run(partition_tokens=pt, out_dtype=out_dtype, **kw), want, ref, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("what", [(math.inf,), (math.nan,), (math.inf, -math.inf, math.nan)], ids=str)
def test_the_same_in_tall_tiles(dtype, what):
    b = Batch([(150, 250), (200, 200), (70, 300)], dtype, H=4, Hkv=2, D=128, seed=40).widen(5000)
    b.max_new = 300
    _, ref, bound = b.reference()
    sprinkle(b, 1, what)
    same_kind(b.run(partition_tokens=-1), expected(b), ref, bound)
    same_kind(b.run(partition_tokens=128), expected(b), ref, bound)


@pytest.mark.parametrize("dtype,D", SHAPES)
@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_rows_that_see_nothing_stay_zero(dtype, D, out_dtype):
    b = Batch([(40, 40)], dtype, H=4, Hkv=2, D=D, seed=13)
    mask = b.tree_masks()
    mask[11] = 0
    b.v[int(b.tables[0, 0]), :, 5] = math.inf
    b.v[int(b.tables[0, 1]), :, 9] = math.nan
    for pt in (-1, 16):
        out = b.run(mask, partition_tokens=pt, out_dtype=out_dtype)
        assert bool((out[11] == 0).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_values_near_the_largest_stay_finite(D, out_dtype):
    """A weight above 1 times such a value passes fp32's range; the average does not.
    Only rows whose weights, taken against their largest, sum to less than 3.9 are
    looked at: outputs are sums in fp32, which 2^126 times 4 passes whatever the order."""
    b = Batch([(40, 300), (1, 900)], "bf16", H=4, Hkv=2, D=D, seed=14, spread=3.0)
    for j in range(300):  # scores grow from the nearest keys on: weights above 1
        b.k[int(b.tables[0, j // 16]), :, j % 16] *= 3 - 2 * j / 300
    b.v.fill_(2.0 ** 126)
    out = b.run(out_dtype=out_dtype, partition_tokens=-1)
    some = 0
    for s, (n, ctx) in enumerate(b.lens):
        j = torch.arange(ctx, device="cuda")
        k = b.k[b.tables[s].long()[j // 16], :, j % 16].double().repeat_interleave(2, 1)
        q = b.q[int(b.starts[s]):int(b.starts[s]) + n].double()
        z = torch.einsum("nhd,jhd->nhj", q, k) * b.scale
        z = z.masked_fill((j > ctx - n + torch.arange(n, device="cuda")[:, None])[:, None], -math.inf)
        few = (z - z.amax(-1, keepdim=True)).exp().sum(-1) < 3.9
        got = out[int(b.starts[s]):int(b.starts[s]) + n][few].double() / 2.0 ** 126
        some += len(got)
        # 300 to 900 weights' roundings, one after another in the sum, at 2^-23 each
        assert bool(((got - 1).abs() <= 900 * 2.0 ** -23 + 2.0 ** -8).all())
    assert some > 10


def time_of(b, **kw):
    ws, out = b.workspace(), torch.empty_like(b.q)
    a, z = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    b.run(out=out, workspace=ws, **kw)
    best = math.inf
    for _ in range(3):
        a.record()
        b.run(out=out, workspace=ws, **kw)
        z.record()
        z.synchronize()
        best = min(best, a.elapsed_time(z))
    return best


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64), ("bf16", 256)])
@pytest.mark.parametrize("where", ["v_inf", "v_nan", "k_nan", "q_nan"])
def test_one_bad_token_does_not_hold_up_a_prompt(dtype, D, where):
    """All later tokens see it, so nearly all results are legitimately not finite.
    (Computing each of them again, key by key, takes hundreds of times as long.)"""
    b = Batch([(2048, 2048)] * 2, dtype, H=8, Hkv=2, D=D, seed=15)
    usual = time_of(b)
    for s in range(2):
        at = (int(b.tables[s, 0]), slice(None), 5, slice(None))
        if where[0] == "q":
            b.q[:] = math.nan
        else:
            (b.v if where[0] == "v" else b.k)[at] = math.inf if "inf" in where else math.nan
    assert time_of(b) < 10 * usual
