"""What the delta rule leaves where a bounded wait runs out: nothing that is wrong and not marked.

A diagnostic on the host leaves out the loads of one chunk in one kind of launch and shortens the waits,
so that CTAs run until there, wait, give up and end by themselves; the context stays usable.  Each entry of
each output must be NaN, or what the undisturbed call gives bit by bit (rows behind a sequence's length are
zero as ever).  The same call afterwards is as before."""
import pytest
import torch

from tests.test_gpu_delta import inputs

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "g", "beta")
LIMIT = 300_000                                       # ns
# whole sequences; segments; pieces (more heads than processors)
SHAPES = {"whole": (3, 300, 4, 2, 128, 64, [300, 0, 65]), "segments": (1, 2000, 2, 1, 128, 128, [1999]),
          "pieces": (40, 1500, 4, 2, 64, 64, [1500, 0, 1, 64, 750, 512, 513, 1499] * 5)}
LAUNCHES = {"prompt": ("PREPARE", "SEGMENTS", "CHAIN"),
            "gradients": ("PREPARE", "SEGMENTS", "CHAIN", "BACK_SEGMENTS", "BACK", "PASS", "ALL")}
CASES = [(w, n, form, chunk) for w, names in LAUNCHES.items() for n in names for form in SHAPES for chunk in (0, 1, 2)
         if (form == "segments" or "SEGMENTS" not in n)
         # (the pass takes 64 value channels of a head at a time: two for a CTA of "whole", no number 2)
         and (n, form, chunk) != ("PASS", "whole", 2)]


@pytest.fixture(scope="module")
def layer():
    from learnable_kv_token_b200 import layer
    return layer


def run(layer, x, do, what):
    args = [x[n] for n in NAMES]
    if what == "prompt":
        return layer.delta_prefill(*args, state=x["state"], lens=x["lens"])
    return layer.delta_backward(*args, do, state=x["state"], lens=x["lens"])


def withheld(layer, x, do, what, launch, chunk):
    try:
        layer.L.lte_gdr_withhold(getattr(layer.L, "LTE_GDR_LAUNCH_" + launch), chunk, LIMIT)
        got = run(layer, x, do, what)
        torch.cuda.synchronize()
    finally:
        layer.L.lte_gdr_withhold(0)
    return got


def same_bits(a, b):
    as_int = {torch.bfloat16: torch.int16, torch.float32: torch.int32}[a.dtype]
    return a.view(as_int) == b.view(as_int)


@pytest.mark.parametrize("what,launch,form,chunk", CASES)
def test_what_is_not_done_is_nan(layer, what, launch, form, chunk):
    *shape, lens = SHAPES[form]
    x = inputs(80, *shape, lens=lens)
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    want = run(layer, x, do, what)
    # the outputs' memory will be some that holds finite values
    del [torch.full_like(t, 7.0) for t in want][:]
    got = withheld(layer, x, do, what, launch, chunk)
    for i, (a, b) in enumerate(zip(got, want)):
        assert (torch.isnan(a) | same_bits(a, b)).all(), i
    assert any(torch.isnan(a).any() for a in got)
    for a, b in zip(run(layer, x, do, what), want):
        assert same_bits(a, b).all()


@pytest.mark.parametrize("launch", ["PREPARE", "CHAIN"])
@pytest.mark.parametrize("shape", [(2, 200, 4, 2, 64, 128), (1, 2000, 2, 1, 128, 128), (40, 1500, 4, 2, 64, 64)], ids=str)
def test_first_chunk_withheld_marks_every_token(layer, launch, shape):
    x = inputs(81, *shape)
    o, S = withheld(layer, x, None, "prompt", launch, 0)
    assert torch.isnan(o).all() and torch.isnan(S).all()


@pytest.mark.parametrize("launch", ["CHAIN", "BACK", "PASS"])
@pytest.mark.parametrize("shape", [(2, 200, 4, 2, 64, 128), (1, 2000, 2, 1, 128, 128), (40, 1500, 4, 2, 64, 64)], ids=str)
def test_first_chunk_withheld_marks_every_gradient(layer, launch, shape):
    """The pass writes no dv and no gradient of the state; the rest of its outputs is all marked, as are
    all that are made from what a chain left."""
    x = inputs(82, *shape)
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    got = withheld(layer, x, do, "gradients", launch, 0)
    for i, a in enumerate(got):
        assert torch.isnan(a).all() or (launch == "PASS" and i in (2, 5)), i
