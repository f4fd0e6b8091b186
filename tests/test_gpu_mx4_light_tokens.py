"""The 4-bit decode where one token has nearly all the weight and a value of nothing, so that the output is made of
tokens far lighter than f16 holds in full.

The weights' product with V runs on halves: P = 2^(logit - m), where the row's largest logit lies 8 or more above m,
times 2^(d - 7) for a scale d = 0 .. 7 steps up its window.  Rounding P and the product costs at most 2^-11 of them,
or, where they are subnormal halves (below 2^-14), 2^-25 each: 2^-24 in all.  A token's contribution is that times a
code of at most 6 and 2^(vref - 127), the window's top, which lies at most three steps above the row's largest scale (the
first token's plus three, or the largest) and at 7 or more.  The denominator is 2^8 or more in the same units, so beside
the relative errors of cache_util an output is off by at most n 2^-32 6 2^(vref - 127)."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from paged_kv_gqa_17_b200 import binding as bd

from . import cache_util as U
from .test_gpu_mx4 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_17_b200 import build

    build.build()
    bd.lib()


@pytest.mark.parametrize("below", [14, 18, 22, 26, 34])
@pytest.mark.parametrize("heavy_at", [0, 3000])
@pytest.mark.parametrize("heavy_scale", [119, 124, 127, 131])
@pytest.mark.parametrize("D", [64, 128])
def test_a_heavy_token_without_a_value(below, heavy_at, heavy_scale, D):
    """Light tokens' weights are around 2^-below of the heavy one's; its V codes are zeros under a scale of its own,
    which is the window's where it comes first."""
    n = 3500
    c = Case([n, 33], 1, 4, D, seed=below + heavy_at)
    c.q[0] = 0
    c.q[0, :, 0] = 1
    c.scale = below * np.log(2) / 24
    scales = np.full(D // 32, 127)
    for t in range(n):
        record = c.pool[c.table[0, t // 16], 0]
        code = c.rng.integers(0, 16, D)
        code[0] = 7 if t == heavy_at else c.rng.choice([0, 1, 2, 9, 10])  # 6, or one of 0, .5, 1, -.5, -1
        C.put(record, t % 16, D, False, code, scales + 2 if t == heavy_at else scales)
        if t == heavy_at:
            C.put(record, t % 16, D, True, np.zeros(D, int), np.full(D // 32, heavy_scale))
        else:
            C.put(record, t % 16, D, True, c.rng.integers(0, 16, D), scales)
    q, pool, table, lens = c.device()
    k, v = U.mx4_rows(c.pool, c.table, c.lens, 0)
    want, w, reach, size = C.attend(c.q[0].double().numpy(), k, v, c.scale, c.G)
    rare = n * 2.0 ** -32 * 6 * 2.0 ** (max(127, heavy_scale) + 3 - 127)
    tol = (U.weight_tolerance(D, c.scale, size)[:, None] + U.F16_HALF) * reach + U.BF16_HALF * np.abs(want) + rare
    if heavy_scale != 127:  # pages with scales outside a window take bf16
        tol += (U.BF16_HALF - U.F16_HALF) * reach
    for blocks in (None, 1):
        plan = bd.plan_mx4(bd.mx4_shape(pool, table, 4), "cuda", scores=True, blocks=blocks)
        scores = torch.from_numpy(c.before).cuda()
        out = bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=scores)[0].double().cpu().numpy()
        assert (np.abs(out - want) <= tol).all(), (float((np.abs(out - want) / tol).max()), float(np.abs(want).max()))
        U.check_scores(scores[0, :, :n].double().cpu().numpy(), c.before[0, :, :n].astype(float), w, size, D, c.scale)
