"""Calls that are given no plan: whose lengths they read, and what becomes of the errors that their kernels meet."""
import pytest
import torch

from paged_kv_gqa_17_b200 import binding as bd

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
