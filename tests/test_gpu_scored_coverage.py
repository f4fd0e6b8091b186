"""The scores of a decode whose plan does not cover its rows, or whose work items are refused: tokens that the call did
not attend to get nothing, above all nothing left over from an earlier call."""
import ctypes

import pytest
import torch

from paged_kv_gqa_17_b200 import binding as bd

from .test_gpu_mx4 import Case as Mx4Case
from .test_gpu_scored import Case, rule

pytestmark = pytest.mark.gpu

ITEM, LEN = 8, 2  # bits of the device error mask


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_17_b200 import build

    build.build()
    bd.lib()


def decode(c, plan):
    """A call on the case's scores; returns (out, scores, error mask)."""
    scores = torch.from_numpy(c.before).cuda()
    out = bd.paged_decode_scored(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, scores, plan=plan)
    return out, scores, bd.workspace_status(plan)


def untouched(c, scores, i, h=slice(None)):
    return (scores[i, h].cpu().numpy() == c.before[i, h]).all()


@pytest.mark.parametrize("G,D", [(4, 128), (1, 64), (16, 64)])
@pytest.mark.parametrize("what", ["begin", "row", "order", "head"])
@pytest.mark.parametrize("which", [0, 1, 2, 3, 7, 8])
@pytest.mark.parametrize("flags", [0, 1])
def test_a_refused_item_leaves_its_pair_without_weights(which, what, flags, G, D):
    """The queue of rows of 100, 30 and 112 tokens at two pages an item: pairs of four, one and four items."""
    c = Case([100, 30, 112], 2, G, D, seed=G)
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", rules=rule(2, 1, 2, flags), scores=True)
    indptr = plan.indptr.tolist()
    assert indptr[:7] == [0, 4, 8, 9, 10, 14, 18]
    out, scores, error = decode(c, plan)
    assert error == 0
    c.check(out, scores)
    item = plan.items[which].tolist()
    bad = {"begin": [item[0], item[1], item[2] + 7, item[3] + 7], "row": [99, item[1], item[2], item[3]],
           "order": [item[0], item[1], item[3] // 16 * 16 + 16, item[2]], "head": [item[0], -1, item[2], item[3]]}[what]
    plan.items[which] = torch.tensor(bad, dtype=torch.int32)
    pair = max(p for p in range(6) if indptr[p] <= which)
    for _ in range(2):  # and again, on the workspace that the refusal left
        _, now, error = decode(c, plan)
        assert error & ITEM
        assert untouched(c, now, pair // 2, pair % 2)
        for other in range(6):
            if other != pair:
                assert torch.equal(now[other // 2, other % 2], scores[other // 2, other % 2]), other


def test_a_pair_whose_items_are_all_refused():
    c = Case([100, 30], 2, 4, 64)
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", rules=rule(2, 1, 2), scores=True)
    _, scores, _ = decode(c, plan)
    plan.items[:4, 0] = 77
    _, now, error = decode(c, plan)
    assert error & ITEM and untouched(c, now, 0, 0)
    assert torch.equal(now[0, 1], scores[0, 1]) and torch.equal(now[1], scores[1])


@pytest.mark.parametrize("rules", [rule(1, 3), rule(1, 1), rule(2, 1, 2), rule(2, 1, 100), rule(1, 2, 0, 1),
                                   rule(2, 1, 1, 1)])
@pytest.mark.parametrize("grown", [1, 16, 37])
def test_rows_that_grew_since_the_plan(rules, grown):
    """Tokens past the plan's are not attended to: no weight for them, the others' weights are among themselves, and
    the call says so."""
    planned = [48, 90, 16]
    c = Case([n + grown for n in planned], 2, 4, 128, seed=grown)
    plan = bd.plan_decode(planned, c.shape(), "cuda", rules=rules, scores=True)
    # what the plan's chunks hold of the longer rows
    S, C = plan.plan.num_splits, plan.plan.chunk_pages
    covered = planned if plan.plan.mode == 2 else [min(n, S * C * 16) for n in c.lens]
    for _ in range(2):
        out, scores, error = decode(c, plan)
        c.check(out, scores, lens=covered)
        assert error == (0 if covered == c.lens else ITEM)


def test_rows_that_grew_after_a_call_that_covered_them():
    c = Case([100, 60], 2, 4, 64)
    long = bd.plan_decode(c.lens, c.shape(), "cuda", rules=rule(2, 1, 2), scores=True)
    decode(c, long)  # leaves logits of every token in the workspace
    short = bd.plan_decode([70, 60], c.shape(), "cuda", rules=rule(2, 1, 2), scores=True)
    assert short.workspace.numel() <= long.workspace.numel()
    short.workspace = long.workspace
    out, scores, error = decode(c, short)
    assert error == ITEM
    c.check(out, scores, lens=[70, 60])


def test_a_row_shorter_than_its_plan_keeps_the_rest_of_its_scores():
    c = Case([100, 60], 2, 4, 64)
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", rules=rule(2, 1, 2), scores=True)
    decode(c, plan)
    c.ld.copy_(torch.tensor([41, 0], dtype=torch.int32))
    _, scores, error = decode(c, plan)
    assert error == 0
    assert (scores[0, :, 41:].cpu().numpy() == c.before[0, :, 41:]).all() and untouched(c, scores, 1)


@pytest.mark.parametrize("first,then", [([100, 30, 112], [20, 112, 7]), ([7, 112, 20], [112, 100, 112])])
def test_a_workspace_that_serves_queues_of_other_lengths(first, then):
    """One workspace, large enough for both queues, whose sections lie elsewhere for each."""
    c = Case([max(x) for x in zip(first, then)], 2, 4, 64, max_pages=7)
    plans = [bd.plan_decode(x, c.shape(), "cuda", rules=rule(2, 1, 1), scores=True) for x in (first, then)]
    shared = max((p.workspace for p in plans), key=lambda w: w.numel())
    for lens, plan in ((first, plans[0]), (then, plans[1]), (then, plans[1])):
        plan.workspace = shared
        c.ld.copy_(torch.tensor(lens, dtype=torch.int32))
        out, scores, error = decode(c, plan)
        assert error == 0
        c.check(out, scores, lens=lens)


def time_out(ws):
    """A wait of a millisecond that nothing satisfies: its bit in the workspace's error word."""
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert bd.lib().pkv_selftest_wait_timeout(ws.data_ptr(), ws.numel(), 1000, stream) == 0


def clear(ws):
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert bd.lib().pkv_workspace_init(ws.data_ptr(), ws.numel(), stream) == 0


def test_nothing_is_added_on_a_workspace_that_timed_out():
    c = Case([100, 30], 2, 4, 64)
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", rules=rule(2, 1, 2), scores=True)
    time_out(plan.workspace)
    _, scores, error = decode(c, plan)
    assert error == 1 and untouched(c, scores, 0) and untouched(c, scores, 1)
    clear(plan.workspace)
    out, scores, error = decode(c, plan)
    assert error == 0
    c.check(out, scores)


def test_nothing_is_added_on_a_workspace_that_timed_out_4_bits():
    c = Mx4Case([100, 30], 2, 4, 64)
    q, pool, table, lens = c.device()
    plan = bd.plan_mx4(bd.mx4_shape(pool, table, 8), "cuda", scores=True)
    for clean in (False, True):
        (clear if clean else time_out)(plan.workspace)
        scores = torch.from_numpy(c.before).cuda()
        out = bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=scores)
        if clean:
            assert bd.workspace_status(plan) == 0
            c.check(out, scores)
        else:
            assert bd.workspace_status(plan) == 1
            assert (scores.cpu().numpy() == c.before).all()


def test_queues_with_gaps_and_missing_pairs_are_reported():
    c = Case([100, 30], 2, 4, 64)
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", rules=rule(2, 1, 2), scores=True)
    assert plan.indptr.tolist() == [0, 4, 8, 9, 10]
    _, scores, _ = decode(c, plan)
    item = plan.items[2].clone()
    plan.items[2, 2] += 16  # its first page belongs to no item now
    _, now, error = decode(c, plan)
    assert error == ITEM and untouched(c, now, 0, 0)
    for i, h in ((0, 1), (1, 0), (1, 1)):
        assert torch.equal(now[i, h], scores[i, h])
    # a queue that ends before the last pair, on a workspace that has seen no other
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", rules=rule(2, 1, 2), scores=True)
    assert plan.items[2].equal(item)
    plan.indptr[4] = 9
    _, now, error = decode(c, plan)
    assert error == ITEM and untouched(c, now, 1, 1) and torch.equal(now[0], scores[0])
