"""Arguments of the 4-bit decode that say "no scores"."""
import pytest
import torch

from paged_kv_gqa_17_b200 import binding as bd

from .test_gpu_mx4 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_17_b200 import build

    build.build()
    bd.lib()


@pytest.mark.parametrize("planned", [True, False])
def test_false_means_no_scores_as_it_does_for_the_plan(planned):
    c = Case([100, 0, 17], 2, 4, 64)
    q, pool, table, lens = c.device()
    plan = bd.plan_mx4(bd.mx4_shape(pool, table, 8), "cuda", scores=False) if planned else None
    out = bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=False)
    c.check(out)
    assert torch.equal(out, bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan))


def test_scores_that_are_no_tensor_are_refused():
    c = Case([100, 0, 17], 2, 4, 64)
    q, pool, table, lens = c.device()
    scored = bd.plan_mx4(bd.mx4_shape(pool, table, 8), "cuda", scores=True)
    for plan in (scored, None):
        with pytest.raises(TypeError):
            bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=True)
    with pytest.raises(ValueError):
        bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=scored, scores=False)
