"""Runs and corners of the cache operators on the GPU: bf16 steps with scores and an eviction between them, graphs that
share a plan, calls without a plan on another stream, batches of nothing, many short rows, wide rows."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from paged_kv_gqa_17_b200 import binding as bd

from . import cache_util as U
from .test_gpu_evict import Case as EvictCase
from .test_gpu_mx4 import Case as Mx4Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_17_b200 import build

    build.build()
    bd.lib()


def test_bf16_steps_scores_and_eviction_together():
    """Steps that append a token and attend with scores, an eviction, and plain and scored steps on what is left."""
    rng = np.random.default_rng(21)
    B, H, G, D, max_pages, budget, recent = 3, 2, 4, 64, 6, 40, 8
    lens_host, scale = [70, 33, 50], D ** -0.5
    table = rng.permutation(B * max_pages).reshape(B, max_pages).astype(np.int32)
    td = torch.from_numpy(table).cuda()
    kv = torch.randn(B * max_pages, 2, H, 16, D, device="cuda").to(torch.bfloat16)  # one combined cache
    k, v = kv[:, 0], kv[:, 1]
    scores = torch.zeros(B, H, max_pages * 16, device="cuda")
    lens = torch.tensor(lens_host, dtype=torch.int32, device="cuda")
    total = np.zeros(scores.shape)
    evict = bd.plan_evict(B, H, max_pages, "cuda")
    for step in range(4):
        for i, n in enumerate(lens.tolist()):
            kv[int(table[i, n // 16]), :, :, n % 16] = torch.randn(2, H, D, device="cuda").to(torch.bfloat16)
        lens += 1
        now = lens.tolist()
        q = torch.randn(B, H * G, D, device="cuda").to(torch.bfloat16)
        plan = bd.plan_decode(now, bd.shape_of(q, k, td, "HND", v), "cuda", scores=True)
        out = bd.paged_decode_scored(q, k, v, td, lens, 16, scale, scores, plan=plan)
        assert bd.workspace_status(plan) == 0
        if step == 3:
            plain = bd.paged_decode(q, k, v, td, lens, 16, scale, seq_lens_host=now)
            assert (plain.double() - out.double()).abs().max() <= 2 ** -7 * out.double().abs().max()
        for i, n in enumerate(now):
            rows = [x[torch.from_numpy(table[i]).long().cuda()].double().cpu().numpy().transpose(1, 0, 2, 3)
                    .reshape(H, -1, D)[:, :n] for x in (k, v)]
            want, w, reach, size = C.attend(q[i].double().cpu().numpy(), *rows, scale, G)
            U.check_out(out[i].double().cpu().numpy(), want, reach, size, D, scale, U.BF16_HALF, (step, i))
            U.check_scores(scores[i].double().cpu().numpy()[:, :n], total[i, :, :n], w, size, D, scale, (step, i))
        if step == 1:
            planes = [x.contiguous().view(torch.int16).cpu().numpy() for x in (k, v)]
            want = C.evict(scores.cpu().numpy(), np.zeros(scores.shape, np.int32), planes, table, now, budget, recent)
            lens = bd.evict_tokens(scores, (k, v), td, lens, budget, recent, plan=evict)
            assert lens.tolist() == want[3] == [40, 35, 40]
            assert (scores.cpu().numpy() == want[0]).all()
            for x, y in zip((k, v), want[2]):
                assert (x.contiguous().view(torch.int16).cpu().numpy() == y).all()
        total = scores.double().cpu().numpy()
    assert bd.workspace_status(evict) == 0


def test_two_graphs_share_a_plan_and_an_eager_call_runs_between():
    c = Mx4Case([300, 17, 90], 2, 4, 128)
    q, pool, table, lens = c.device()
    plan = bd.plan_mx4(bd.mx4_shape(pool, table, 8), "cuda", scores=True)
    scores = torch.from_numpy(c.before).cuda()
    outs = [torch.empty_like(q) for _ in range(2)]
    graphs = []
    for out in outs:
        bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=scores, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=scores, out=out)
        graphs.append(g)
    for turn in (0, 1, 1, 0):
        scores.copy_(torch.from_numpy(c.before))
        outs[turn].zero_()
        graphs[turn].replay()
        torch.cuda.synchronize()
        c.check(outs[turn], scores)
        scores.copy_(torch.from_numpy(c.before))
        c.check(bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=scores), scores)


def test_calls_without_a_plan_on_another_stream():
    c = Mx4Case([300, 17, 90], 2, 4, 64)
    q, pool, table, lens = c.device()
    scores = torch.from_numpy(c.before).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        scores_now = scores.clone()
        side.wait_stream(torch.cuda.current_stream())
        out = bd.mx4_decode(q, pool, table, lens, 16, c.scale, scores=scores_now, stream=side)
        torch.full((1 << 20,), 77, dtype=torch.uint8, device="cuda")  # what takes freed memory of this stream
        side.synchronize()
        c.check(out, scores_now)
    k = torch.randn(3, 2, 64, device="cuda").to(torch.bfloat16)
    side.wait_stream(torch.cuda.current_stream())
    at = torch.tensor([2, 3, 4], dtype=torch.int32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    bd.mx4_append(k, k, pool, table, at, stream=side)
    gk, gv = bd.mx4_read(pool, table, at, 3, stream=side)
    side.synchronize()
    want = C.values(*C.quantise(k.double().cpu().numpy()))
    assert (gk.double().cpu().numpy() == want).all() and (gv.double().cpu().numpy() == want).all()


def test_batches_of_nothing():
    c = Mx4Case([30, 17], 2, 4, 64)
    q, pool, table, lens = c.device()
    assert bd.mx4_decode(q[:0], pool, table[:0], lens[:0], 16, 1.0).shape == (0, 8, 64)
    before = pool.clone()
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    ind = torch.zeros(3, dtype=torch.int32, device="cuda")
    bd.mx4_append(none, none, pool, table, lens, indptr=ind)
    assert [x.shape for x in bd.mx4_read(pool, table, lens, 0, indptr=ind)] == [(0, 2, 64)] * 2
    e = EvictCase([30, 17], 2, (16,))
    scores, positions, planes, table, lens = e.device()
    assert bd.evict_tokens(scores[:0], planes, table[:0], lens[:0], 4, 2, positions=positions[:0]).shape == (0,)
    torch.cuda.synchronize()
    assert torch.equal(pool, before) and (planes[0].cpu().numpy() == e.planes[0]).all()


@pytest.mark.parametrize("G,D", [(4, 128), (16, 64)])
def test_many_short_rows(G, D):
    """Runs of a page or less, pairs that begin inside a stage, empty rows between them."""
    lens = [int(x) for x in np.random.default_rng(31).choice([0, 1, 5, 15, 16, 17, 31, 32, 33, 47, 48, 49, 80], 150)]
    c = Mx4Case(lens, 3, G, D, seed=G)
    c.run(True)
    c.run(False, 7)


def test_a_plan_of_another_device_is_refused():
    c = Mx4Case([30, 17], 2, 4, 64)
    q, pool, table, lens = c.device()
    plan = bd.plan_mx4(bd.mx4_shape(pool, table, 8), "cuda")
    plan.workspace = plan.workspace.cpu()
    with pytest.raises(ValueError):
        bd.mx4_decode(q, pool, table, lens, 16, 1.0, plan=plan)
    e = EvictCase([30, 17], 2, (16,))
    scores, _, planes, table, lens = e.device()
    evict = bd.plan_evict(2, 2, e.max_pages, "cuda")
    evict.workspace = evict.workspace.cpu()
    with pytest.raises(ValueError):
        bd.evict_tokens(scores, planes, table, lens, 4, 2, plan=evict)


@pytest.mark.parametrize("widths", [(4096,), (4096,) * 8, (4095,), (4095, 4096, 8), (1,)])
def test_eviction_of_rows_wider_than_the_block(widths):
    EvictCase([150, 40, 99], 1, widths, seed=len(widths)).run(64, 40)


@pytest.mark.parametrize("n,budget,recent", [(20000, 9000, 4000), (20000, 19999, 19000), (17000, 300, 0)])
def test_long_rows_and_windows(n, budget, recent):
    for kind in ("exp", "equal"):
        c = EvictCase([n, 50], 1, (16, 4), kind, seed=n)
        c.run(budget, recent)
