"""Evictions of the same rows under block tables of every width: which variant runs goes by the table's width, what it
does must not."""
import pytest
import torch

from paged_kv_gqa_17_b200 import binding as bd

from .test_gpu_evict import Case

pytestmark = pytest.mark.gpu

# on both sides of where a block stops selecting for its cluster, and for itself; and wide tables
CAPACITIES = [2064, 6144, 6160, 8192, 14336, 14352, 16384, 16400, 32768, 131072]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_17_b200 import build

    build.build()
    bd.lib()


@pytest.mark.parametrize("B,H", [(2, 2), (5, 8), (9, 8), (19, 8)])  # clusters of eight, four and two, and no cluster
def test_tables_wider_than_the_rows(B, H):
    lens = [2064 - 7 * i if i % 3 else 40 * i for i in range(B)]
    c = Case(lens, H, (16, 4), "few", seed=B)
    budget, recent = 1500, 100
    want = c.want(budget, recent)
    scores, positions, planes, table, lens_d = c.device()
    tokens = scores.shape[2]
    for capacity in CAPACITIES:
        wide = torch.full((B, capacity // 16), 2 ** 30, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        s = torch.full((B, H, capacity), -3.0, device="cuda")
        s[:, :, :tokens] = scores
        pos = torch.full((B, H, capacity), -3, dtype=torch.int32, device="cuda")
        pos[:, :, :tokens] = positions
        now = [p.clone() for p in planes]
        plan = bd.plan_evict(B, H, capacity // 16, "cuda")
        new = bd.evict_tokens(s, now, wide, lens_d, budget, recent, positions=pos, plan=plan)
        assert bd.workspace_status(plan) == 0 and new.tolist() == want[3], capacity
        assert (s[:, :, :tokens].cpu().numpy() == want[0]).all() and (s[:, :, tokens:] == -3.0).all(), capacity
        assert (pos[:, :, :tokens].cpu().numpy() == want[1]).all() and (pos[:, :, tokens:] == -3).all(), capacity
        for p, w in zip(now, want[2]):
            assert (p.cpu().numpy() == w).all(), capacity


@pytest.mark.parametrize("n", [6144, 6145, 14336, 14337])
@pytest.mark.parametrize("kind", ["exp", "odd"])
def test_rows_that_fill_a_variants_last_slot(n, kind):
    for rows in (1, 149):
        c = Case([n] + [30] * (rows - 1), 1, (8,), kind, seed=n)
        c.run(n - 1, 0)
        c.run(n // 3, n // 9)


def test_rows_above_and_below_the_budget_side_by_side():
    Case([7000, 10, 6999, 500], 3, (64,), seed=2).run(501, 77)


def test_planes_that_share_memory_are_refused():
    c = Case([100, 40], 2, (16, 32))
    scores, positions, planes, table, lens = c.device()

    def call(p, **kw):
        return bd.evict_tokens(scores, p, table, lens, 20, 4, **kw)

    for p in ([planes[0], planes[0]], [planes[0], planes[1], planes[0].view(torch.int32)],
              [planes[1][..., :20], planes[1][..., 19:]]):
        with pytest.raises(ValueError):
            call(p)
    with pytest.raises(ValueError):
        call(planes, positions=scores.view(torch.int32))
    # halves of one array share none, whichever comes first
    want = c.want(20, 4)
    call([planes[1][..., 16:], planes[0], planes[1][..., :16]])
    for p, w in zip(planes, want[2]):
        assert (p.cpu().numpy() == w).all()
