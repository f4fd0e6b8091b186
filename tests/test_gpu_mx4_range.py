"""The 4-bit decode over the whole range of its numbers: keys and queries whose magnitudes cancel."""
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


def key_scales(c):
    """The K scale bytes [pages][H][16][D/32] of a case's pool, as a view."""
    pages, H, _ = c.pool.shape
    return c.pool[:, :, 16 * c.D:16 * c.D + c.D // 2].reshape(pages, H, 16, c.D // 32)


def set_key_scales(c, scales):
    flat = scales.reshape(c.pool.shape[0], c.H, -1)
    c.pool[:, :, 16 * c.D:16 * c.D + c.D // 2] = flat


@pytest.mark.parametrize("byte", [1, 2, 16, 40, 64, 100, 160, 200, 219, 226, 232, 233, 234, 236, 240, 246, 252])
@pytest.mark.parametrize("G,D", [(4, 128), (4, 64), (16, 128)])
def test_logits_of_a_few_units_whatever_the_keys_scale(byte, G, D):
    """Keys of 2^(byte - 127) times a few, queries as much smaller (or larger)."""
    c = Case([1, 40, 700, 0, 33], 2, G, D, seed=byte + G)
    s = key_scales(c).astype(int)
    set_key_scales(c, np.where(s == 255, 255, np.clip(s - 126 + byte, 1, 252)).astype(np.uint8))
    c.q = torch.from_numpy(c.q.double().numpy() * 2.0 ** (126 - byte)).to(torch.bfloat16)
    c.run(False)
    c.run(True, 3)


def test_keys_of_every_magnitude_in_one_row():
    """Ordinary queries: the keys' scales run over the whole range, the largest logits decide."""
    c = Case([500, 20, 90], 2, 4, 128, seed=5)
    s = key_scales(c)
    set_key_scales(c, np.where(s == 255, 255, c.rng.integers(1, 241, s.shape)).astype(np.uint8))
    q, pool, table, lens = c.device()
    plan = bd.plan_mx4(bd.mx4_shape(pool, table, 8), "cuda", scores=True)
    scores = torch.from_numpy(c.before).cuda()
    out = bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=scores).double().cpu().numpy()
    assert bd.workspace_status(plan) == 0
    for i, n in enumerate(c.lens):
        k, v = U.mx4_rows(c.pool, c.table, c.lens, i)
        want, w, reach, size = C.attend(c.q[i].double().numpy(), k, v, c.scale, c.G)
        # one token has all the weight where the largest two logits of every head lie further apart than their errors
        x = np.einsum("hnd,hgd->hgn", k, c.q[i].double().numpy().reshape(2, 4, -1)) * c.scale
        top = np.sort(x, -1)[..., -2:]
        assert (top[..., 1] - top[..., 0] > 2 * U.logit_error(c.D, c.scale, size.reshape(2, 4)) + 100).all()
        U.check_out(out[i], want, reach, np.zeros_like(size), c.D, c.scale, U.F16_HALF, i)
        U.check_scores(scores[i, :, :n].double().cpu().numpy(), c.before[i, :, :n].astype(float), w,
                       np.zeros_like(size), c.D, c.scale, i)


def test_one_key_of_an_extreme_scale_in_an_ordinary_row():
    """Tokens whose keys are huge where their codes are zero, and tiny elsewhere: scales alone must not decide."""
    c = Case([300, 33], 2, 4, 128, seed=6)
    s = key_scales(c).copy()
    for t in (0, 17, 40, 299):
        page, slot = c.table[0, t // 16], t % 16
        for h in range(2):
            code, scale = C.get(c.pool[page, h], 128, False)
            code[slot, 32:64] = 0
            s[page, h, slot, 1] = 252
            s[page, h, slot, 2] = 1
            keep = c.pool[page, h].copy()
            C.put(keep, slot, 128, False, code[slot], s[page, h, slot])
            c.pool[page, h] = keep
    c.run(True)


@pytest.mark.parametrize("exponent", [-133, -130, -126, -118, -110])
def test_queries_down_to_the_smallest(exponent):
    """bf16's subnormal queries included, against keys as large as the format has."""
    c = Case([90, 1, 33], 2, 4, 128, seed=200 + exponent)
    s = key_scales(c).astype(int)
    byte = min(252, 126 - exponent)
    set_key_scales(c, np.where(s == 255, 255, np.clip(s - 126 + byte, 1, 252)).astype(np.uint8))
    c.q = torch.from_numpy(c.q.double().numpy() * 2.0 ** exponent).to(torch.bfloat16)
    c.run(True)


def test_products_that_overflow_to_minus_infinity():
    """The dot product itself leaves fp32, as in the bf16 decode's test."""
    c = Case([40, 20], 1, 2, 64)
    for t in range(40):
        C.put(c.pool[c.table[0, t // 16], 0], t % 16, 64, False, np.full(64, 15), np.array([252, 252]))  # -6 2^125
    c.q[0] = 3.0e38
    q, pool, table, lens = c.device()
    plan = bd.plan_mx4(bd.mx4_shape(pool, table, 2), "cuda", scores=True)
    scores = torch.from_numpy(c.before).cuda()
    out = bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=scores)
    assert (out[0] == 0).all() and torch.isfinite(out).all()
    assert (scores[0].cpu().numpy() == c.before[0]).all() and torch.isfinite(scores).all()
