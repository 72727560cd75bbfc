"""Equal calls give equal bits, whatever other calls leave behind in between."""
import pytest
import torch

from tests.extend_helpers import Batch, slopes
from tests.test_gpu_extend_caps import LARGE, leave_in_shared_memory

pytestmark = pytest.mark.gpu

FORMS = ["plain", "alibi", "cap", "cap_alibi", "window", "prefix", "tree", "tree_cap"]


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f16", 128), ("bf16", 256), ("f32", 64)])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("pt", [0, 64])
def test_every_form(dtype, D, form, pt):
    b = Batch([(1, 3000), (64, 2000), (300, 700), (1, 1), (7, 90)], dtype, H=8, Hkv=2, D=D, seed=28)
    kw = dict(partition_tokens=pt, workspace=b.workspace(pt))
    if "cap" in form:
        kw["softcap"] = 20.0
    if "alibi" in form:
        kw["alibi_slopes"] = slopes(8)
    if form == "window":
        kw["window"] = 200
    if form == "prefix":
        kw["prefix_lens"] = torch.tensor([5, 1990, 400, 0, 90], dtype=torch.int32, device="cuda")
    if "tree" in form:
        kw["mask"] = b.tree_masks()
    first = b.run(**kw)
    for i in range(4):
        if dtype != "f32":
            leave_in_shared_memory(dtype, D, (0.0, LARGE[dtype])[i % 2])
        if kw["workspace"] is not None:
            kw["workspace"].view(torch.float32).fill_(float("nan"))
        assert torch.equal(b.run(**kw), first)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tall_tiles(dtype):
    b = Batch([(300, 700), (1, 4500), (130, 130)], dtype, H=8, Hkv=2, D=128, seed=29).widen(5000)
    for mask in (None, b.tree_masks()):
        for pt in (-1, 256):
            first = b.run(mask, partition_tokens=pt)
            for _ in range(3):
                leave_in_shared_memory(dtype, 128, LARGE[dtype])
                assert torch.equal(b.run(mask, partition_tokens=pt), first)
