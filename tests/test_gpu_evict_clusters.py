"""Evictions by clusters of every size, in batches of several times what runs at once, so that the blocks of a cluster
start while others are busy: bit for bit, over and over."""
import pytest
import torch

from paged_kv_gqa_17_b200 import binding as bd

from .test_gpu_evict import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_17_b200 import build

    build.build()
    bd.lib()


@pytest.mark.parametrize("rows", [1, 19, 37, 50, 74, 100, 148, 160])
@pytest.mark.parametrize("capacity", [300, 600, 1100, 2100, 4100])
def test_every_cluster_size(rows, capacity):
    """One block to eight select for each other; rows within the budget leave at once, beside rows that work."""
    lens = [capacity - 37 * (i % 8) if i % 5 else i % 60 for i in range(rows)]
    c = Case(lens, 1, (16, 4), "exp" if rows % 2 else "few", seed=rows, max_pages=-(-capacity // 16))
    state = c.device()
    plan = bd.plan_evict(rows, 1, c.max_pages, "cuda")
    want = c.want(180, 33)
    for _ in range(6):
        scores, positions, planes, table, lens_d = (x.clone() if isinstance(x, torch.Tensor) else [p.clone() for p in x]
                                                    for x in state)
        new = bd.evict_tokens(scores, planes, table, lens_d, 180, 33, positions=positions, plan=plan)
        assert new.tolist() == want[3]
        assert (scores.cpu().numpy() == want[0]).all() and (positions.cpu().numpy() == want[1]).all()
        for p, w in zip(planes, want[2]):
            assert (p.cpu().numpy() == w).all()
    assert bd.workspace_status(plan) == 0


def test_evictions_behind_kernels_that_hold_the_gpu():
    """Four streams of evictions at once, each with a plan of its own: clusters wait for room block by block."""
    cases = [Case([5000 - 100 * i, 3000, 64], 8, (64, 64), seed=i) for i in range(4)]
    state = [c.device() for c in cases]
    plans = [bd.plan_evict(3, 8, c.max_pages, "cuda") for c in cases]
    outs = [torch.empty(3, dtype=torch.int32, device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for (scores, positions, planes, table, lens), plan, out, st in zip(state, plans, outs, streams):
        bd.evict_tokens(scores, planes, table, lens, 1700, 164, positions=positions, plan=plan, out=out, stream=st)
    torch.cuda.synchronize()
    for c, (scores, positions, planes, _, _), out in zip(cases, state, outs):
        c.check((scores, positions, planes, out), 1700, 164)
