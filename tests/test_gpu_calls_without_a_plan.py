"""Calls that are given no plan: whose lengths they read, and what becomes of the errors that their kernels meet."""
import pytest
import torch

from paged_kv_gqa_17_b200 import binding as bd

from .test_gpu_mx4 import Case as Mx4Case
from .test_gpu_scored import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_17_b200 import build

    build.build()
    bd.lib()


@pytest.mark.parametrize("scored", [True, False])
def test_lengths_are_read_in_the_order_of_the_calls_stream(scored):
    """The lengths are written on the call's stream, behind a tenth of a second of waiting."""
    c = Case([100, 33, 64], 2, 4, 128)
    c.ld = torch.ones(3, dtype=torch.int32, device="cuda")
    late = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    scores = torch.from_numpy(c.before).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        c.ld.copy_(late)
    if scored:
        out = bd.paged_decode_scored(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, scores, stream=side)
    else:
        out = bd.paged_decode(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, stream=side)
    torch.cuda.synchronize()
    if not scored:  # the scored decode adds its own weights to compare with
        bd.paged_decode_scored(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, scores)
    c.check(out, scores)


@pytest.fixture()
def clean():
    bd.unplanned_status()
    yield
    assert bd.unplanned_status() == 0


LEN, PAGE = 2, 4  # bits of the device error mask


def test_errors_of_appends_and_reads(clean):
    c = Mx4Case([30, 17], 2, 4, 64)
    q, pool, table, lens = c.device()
    kv = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([3, 10 ** 6], dtype=torch.int32, device="cuda")
    bd.mx4_append(kv, kv, pool, table, at)
    assert bd.unplanned_status() == LEN and bd.unplanned_status() == 0
    bd.mx4_read(pool, table, at, 2)
    assert bd.unplanned_status() == LEN
    bad = table.clone()
    bad[1, 0] = -1
    at[1] = 4
    bd.mx4_append(kv, kv, pool, bad, at)
    bd.mx4_read(pool, bad, torch.full_like(at, -1), 2)
    assert bd.unplanned_status() == LEN | PAGE
    bd.mx4_append(kv, kv, pool, table, at)  # nothing wrong: the fixture looks


def test_errors_of_decodes_and_evictions(clean):
    c = Mx4Case([30, 17], 2, 4, 64)
    q, pool, table, lens = c.device()
    bad = table.clone()
    bad[0, 1] = 10 ** 6
    bd.mx4_decode(q, pool, bad, lens, 16, c.scale)
    assert bd.unplanned_status() == PAGE
    scores = torch.from_numpy(c.before).cuda()
    bd.mx4_decode(q, pool, table, torch.tensor([5, -1], dtype=torch.int32, device="cuda"), 16, c.scale, scores=scores)
    assert bd.unplanned_status() == LEN
    bd.evict_tokens(scores, bd.mx4_planes(pool), table, torch.tensor([10 ** 6, 3], dtype=torch.int32, device="cuda"), 8, 2)
    assert bd.unplanned_status() == LEN
    d = Case([40, 17], 2, 4, 64)
    d.td[1, 1] = -7
    scores = torch.from_numpy(d.before).cuda()
    bd.paged_decode_scored(d.qd, d.kd, d.vd, d.td, d.ld, 16, d.scale, scores)
    assert bd.unplanned_status() == PAGE
    bd.paged_decode(d.qd, d.kd, d.vd, d.td, d.ld, 16, d.scale)
    assert bd.unplanned_status() == PAGE
    # a plan's errors are the plan's
    plan = bd.plan_decode(d.lens, d.shape(), "cuda")
    bd.paged_decode(d.qd, d.kd, d.vd, d.td, d.ld, 16, d.scale, plan=plan)
    assert bd.workspace_status(plan) == PAGE and bd.unplanned_status() == 0


def test_errors_on_another_stream_and_in_a_replayed_graph(clean):
    c = Mx4Case([30, 17], 2, 4, 64)
    q, pool, table, lens = c.device()
    kv = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([3, 10 ** 6], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bd.mx4_append(kv, kv, pool, table, at, stream=side)
    assert bd.unplanned_status(side) == LEN
    at[1] = 3
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bd.mx4_append(kv, kv, pool, table, at)
    g.replay()
    assert bd.unplanned_status() == 0
    at[1] = -1
    for _ in range(2):
        g.replay()
        assert bd.unplanned_status() == LEN
