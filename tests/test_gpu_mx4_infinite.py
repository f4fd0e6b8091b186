"""Logits of -inf in the 4-bit decode: no weight, as in the bf16 decode."""
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


def overflow(c, i, tokens, heads):
    """Logits of row i's first `tokens` tokens become -inf for the query heads in `heads` (products of magnitudes 2^100
    and 2^100); those heads' later logits, and all the other heads' logits, stay ordinary."""
    assert c.H == 1
    q = c.q[i].double().numpy()
    s = key_scales(c).astype(int)
    live = s != 255
    big = np.zeros_like(live)
    for t in range(min(tokens, c.lens[i])):
        big[c.table[i, t // 16], 0, t % 16] = True
        record = c.pool[c.table[i, t // 16], 0]
        code, scale = C.get(record, c.D, False)
        C.put(record, t % 16, c.D, False, np.full(c.D, 8 | 5), scale[t % 16])  # -3 in every dim
    mine = np.zeros_like(live)
    mine[c.table[i, :-(-c.lens[i] // 16)]] = True
    set_key_scales(c, np.where(live & mine, np.where(big, 227, 27), s).astype(np.uint8))
    for g in range(c.G):
        q[g] = np.abs(q[g]) * 2.0 ** 100 + 2.0 ** 98 if g in heads else q[g] * 2.0 ** -100
    c.q[i] = torch.from_numpy(q).to(torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 20, 700])
@pytest.mark.parametrize("heads", [[0, 1, 2, 3], [1], [0, 3]])
def test_a_row_whose_logits_are_all_minus_infinity_gets_no_weight(n, heads, D):
    c = Case([n, 20], 1, 4, D, seed=n)
    overflow(c, 0, n, heads)
    q, pool, table, lens = c.device()
    for blocks in (None, 1):
        plan = bd.plan_mx4(bd.mx4_shape(pool, table, 4), "cuda", scores=True, blocks=blocks)
        scores = torch.from_numpy(c.before).cuda()
        out = bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=scores)
        assert bd.workspace_status(plan) == 0
        assert (out[0, heads] == 0).all() and torch.isfinite(out).all() and torch.isfinite(scores).all()
        if len(heads) == 4:
            assert (scores[0].cpu().numpy() == c.before[0]).all()
        # the other heads' weights are all that is added
        added = scores[0, 0].double().cpu().numpy() - c.before[0, 0]
        assert abs(added.sum() - (4 - len(heads))) < 1e-3
        unscored = bd.mx4_decode(q, pool, table, lens, 16, c.scale)
        assert (unscored[0, heads] == 0).all() and torch.isfinite(unscored).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens", [1, 16, 31, 32, 33, 64, 250])
@pytest.mark.parametrize("heads", [[0, 1, 2, 3], [2]])
def test_a_row_that_begins_with_logits_of_minus_infinity(tokens, heads, D):
    """What follows has all the weight."""
    n = 400
    c = Case([n, 20], 1, 4, D, seed=tokens)
    overflow(c, 0, tokens, heads)
    q, pool, table, lens = c.device()
    k, v = U.mx4_rows(c.pool, c.table, c.lens, 0)
    heads_q = c.q[0].double().numpy()
    want, weights, reach, size = np.zeros((4, D)), np.zeros((1, n)), np.zeros((4, D)), np.zeros(4)
    for g in range(4):
        begin = tokens if g in heads else 0
        o, w, r, z = C.attend(heads_q[g:g + 1], k[:, begin:], v[:, begin:], c.scale, 1)
        want[g], reach[g], size[g] = o[0], r[0], z[0]
        weights[:, begin:] += w
    for blocks in (None, 1, 2):
        plan = bd.plan_mx4(bd.mx4_shape(pool, table, 4), "cuda", scores=True, blocks=blocks)
        scores = torch.from_numpy(c.before).cuda()
        out = bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=scores)
        assert bd.workspace_status(plan) == 0
        U.check_out(out[0].double().cpu().numpy(), want, reach, size, D, c.scale, U.F16_HALF, blocks)
        U.check_scores(scores[0, :, :n].double().cpu().numpy(), c.before[0, :, :n].astype(float), weights, size, D,
                       c.scale, blocks)
    out = bd.mx4_decode(q, pool, table, lens, 16, c.scale)
    U.check_out(out[0].double().cpu().numpy(), want, reach, size, D, c.scale, U.F16_HALF)
