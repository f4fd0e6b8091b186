"""The 4-bit paged cache on the GPU: tokens quantised into it (byte for byte), read back (exactly) and attended,
against the fp64 oracle; and a run of the cache operators together."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from paged_kv_gqa_17_b200 import binding as bd

from . import cache_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_17_b200 import build

    build.build()
    bd.lib()


# ---------------------------------------------------------------------------
# tokens in and out

def tokens(rng, n, H, D):
    """bf16 values over many magnitudes, with blocks of zeros, subnormals, huge values, infinities and NaN."""
    x = rng.standard_normal((n, H, D)) * 2.0 ** rng.integers(-20, 20, (n, H, D // 32)).repeat(32, -1)
    flat = x.reshape(-1, 32)
    kinds = rng.integers(0, 40, len(flat))
    flat[kinds == 0] = 0.0
    flat[kinds == 1] *= 1e-39 / 2.0 ** -20
    flat[kinds == 2] = rng.choice([3.0e38, -3.0e38, 1e38], (int((kinds == 2).sum()), 32))
    flat[kinds == 3, 7] = np.inf
    flat[kinds == 4, 31] = -np.inf
    flat[kinds == 5, 0] = np.nan
    flat[kinds == 6] = rng.choice([0.0, -0.0, 5.0, 2.5, -3.5, 0.25, 0.75, -1.25], (int((kinds == 6).sum()), 32))
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def stored(pool, k, v, table, starts, indptr):
    """The pool after an append, and the values of its tokens (zeros for skipped ones)."""
    pool = pool.copy()
    n, H, D = k.shape
    got = [np.zeros((n, H, D)), np.zeros((n, H, D))]
    for i, start in enumerate(starts):
        for j in range(indptr[i], indptr[i + 1]):
            at = start + j - indptr[i]
            if at < 0 or at >= table.shape[1] * 16 or not 0 <= table[i, at // 16] < len(pool):
                continue
            for is_v, x in enumerate((k, v)):
                code, scale = C.quantise(x[j].double().numpy())
                got[is_v][j] = C.values(code, scale)
                for h in range(H):
                    C.put(pool[table[i, at // 16], h], at % 16, D, bool(is_v), code[h], scale[h])
    return pool, got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,starts,counts", [(1, [0], [1]), (3, [0, 5, 16, 31, 100], [1, 0, 40, 17, 3]),
                                             (8, [7, 0], [0, 130]), (2, [3] * 40, [1] * 40)])
def test_append_and_read(D, H, starts, counts):
    rng = np.random.default_rng(D + H)
    lens = [s + c for s, c in zip(starts, counts)]
    max_pages = max(-(-n // 16) for n in lens) + 1
    table, pages = U.scattered_table(rng, lens, max_pages)
    indptr = np.concatenate([[0], np.cumsum(counts)])
    n = int(indptr[-1])
    k, v = tokens(rng, n, H, D), tokens(rng, n, H, D)
    before = rng.integers(0, 256, (pages, H, 17 * D)).astype(np.uint8)
    pool, td = torch.from_numpy(before).cuda(), torch.from_numpy(table).cuda()
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    plan = bd.plan_mx4(bd.mx4_shape(pool, td), "cuda")
    ind = torch.from_numpy(indptr.astype(np.int32)).cuda()
    if counts == [1] * len(counts):
        ind = None
    bd.mx4_append(k.cuda(), v.cuda(), pool, td, start, plan=plan, indptr=ind)
    gk, gv = bd.mx4_read(pool, td, start, n, plan=plan, indptr=ind)
    torch.cuda.synchronize()
    assert bd.workspace_status(plan) == 0
    want_pool, (wk, wv) = stored(before, k, v, table, starts, indptr)
    for p, q in zip(bd.mx4_planes(pool.cpu()), bd.mx4_planes(torch.from_numpy(want_pool))):
        assert torch.equal(p, q)
    for got, want in ((gk, wk), (gv, wv)):
        assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("D,H,counts", [(128, 7, [1501, 0, 700]), (64, 15, [33, 1931])])
def test_prompts_long_enough_for_several_rounds(D, H, counts):
    """More rows than a full GPU takes at one each, the last pass of a warp cut off."""
    rng = np.random.default_rng(D)
    starts = [3, 5, 20][:len(counts)]
    lens = [s + c for s, c in zip(starts, counts)]
    table, pages = U.scattered_table(rng, lens, max(-(-n // 16) for n in lens))
    indptr = np.concatenate([[0], np.cumsum(counts)])
    n = int(indptr[-1])
    assert n * H * D // 256 > 148 * 64 * 3 // 4 and n * H % (1024 // D) != 0
    k, v = tokens(rng, n, H, D), tokens(rng, n, H, D)
    before = rng.integers(0, 256, (pages, H, 17 * D)).astype(np.uint8)
    pool, td = torch.from_numpy(before).cuda(), torch.from_numpy(table).cuda()
    start, ind = (torch.from_numpy(np.asarray(x, np.int32)).cuda() for x in (starts, indptr))
    plan = bd.plan_mx4(bd.mx4_shape(pool, td), "cuda")
    bd.mx4_append(k.cuda(), v.cuda(), pool, td, start, plan=plan, indptr=ind)
    gk, gv = bd.mx4_read(pool, td, start, n, plan=plan, indptr=ind)
    assert bd.workspace_status(plan) == 0
    want, (wk, wv) = stored(before, k, v, table, starts, indptr)
    assert (pool.cpu().numpy() == want).all()
    for got, w in ((gk, wk), (gv, wv)):
        assert np.array_equal(got.double().cpu().numpy(), w, equal_nan=True)


def test_append_strided_inputs_and_pool():
    rng = np.random.default_rng(1)
    H, D, n = 2, 128, 21
    table, pages = U.scattered_table(rng, [n + 4], 3)
    qkv = tokens(rng, n, 3 * H + 1, D + 32).cuda()           # a fused projection's output
    k, v = qkv[:, 1:1 + H, :D], qkv[:, 1 + H:1 + 2 * H, :D]
    wide = torch.full((pages, H + 1, 17 * D + 32), 9, dtype=torch.uint8, device="cuda")
    pool = wide[:, :H, :17 * D]
    td = torch.from_numpy(table).cuda()
    start = torch.tensor([4], dtype=torch.int32, device="cuda")
    ind = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    bd.mx4_append(k, v, pool, td, start, indptr=ind)
    gk, gv = bd.mx4_read(pool, td, start, n, indptr=ind)
    want, (wk, wv) = stored(np.full((pages, H, 17 * D), 9, np.uint8), k.cpu(), v.cpu(), table, [4], [0, n])
    assert (pool.cpu().numpy() == want).all()
    assert np.array_equal(gk.double().cpu().numpy(), wk, equal_nan=True)
    assert np.array_equal(gv.double().cpu().numpy(), wv, equal_nan=True)
    pool.fill_(9)
    assert (wide == 9).all()


def test_tokens_without_a_place_are_skipped():
    rng = np.random.default_rng(2)
    H, D = 2, 64
    table, pages = U.scattered_table(rng, [32, 32], 2)
    td = torch.from_numpy(table).cuda()
    k, v = tokens(rng, 12, H, D), tokens(rng, 12, H, D)
    indptr = np.array([0, 4, 9])  # tokens 9 to 11 belong to no row
    for starts, bad_page, error in (([0, 10], None, 0), ([30, 10], None, 2), ([-2, 10], None, 2), ([0, 10], (1, 0), 4)):
        tab = table.copy()
        if bad_page:
            tab[bad_page] = -1
        td = torch.from_numpy(tab).cuda()
        before = rng.integers(0, 256, (pages, H, 17 * D)).astype(np.uint8)
        pool = torch.from_numpy(before).cuda()
        start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        ind = torch.from_numpy(indptr.astype(np.int32)).cuda()
        plan = bd.plan_mx4(bd.mx4_shape(pool, td), "cuda")
        out = tuple(torch.full((12, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        bd.mx4_append(k.cuda(), v.cuda(), pool, td, start, plan=plan, indptr=ind)
        bd.mx4_read(pool, td, start, 12, plan=plan, indptr=ind, out=out)
        assert bd.workspace_status(plan) == error
        want, (wk, wv) = stored(before, k, v, tab, starts, indptr)
        assert (pool.cpu().numpy() == want).all()
        for got, w in zip(out, (wk, wv)):
            assert np.array_equal(got.double().cpu().numpy(), w, equal_nan=True)


# ---------------------------------------------------------------------------
# decode

class Case:
    def __init__(self, lens, H, G, D, seed=1, spread=0, zeros=0.0, max_pages=None, poison=True, q_scale=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.H, self.G, self.D = rng, lens, H, G, D
        self.max_pages = max_pages or max(1, max(-(-n // 16) for n in lens))
        self.table, pages = U.scattered_table(rng, lens, self.max_pages)
        self.pool = U.mx4_pool(rng, pages, H, D, spread, zeros)
        if poison:
            U.poison_tails(self.pool, self.table, lens)
        # logits of a few units, whatever the scales: q shrinks as the keys' scales grow
        self.scale = D ** -0.5 * 0.4 * 2.0 ** -spread
        self.q = torch.from_numpy(rng.standard_normal((len(lens), H * G, D)) * q_scale).to(torch.bfloat16)
        self.before = rng.random((len(lens), H, self.max_pages * 16)).astype(np.float32)

    def device(self):
        return (self.q.cuda(), torch.from_numpy(self.pool).cuda(), torch.from_numpy(self.table).cuda(),
                torch.tensor(self.lens, dtype=torch.int32, device="cuda"))

    def check(self, out, scores=None, lens=None, p_step=U.F16_HALF, what=""):
        out = out.double().cpu().numpy()
        lens = lens or self.lens
        for i, n in enumerate(lens):
            k, v = U.mx4_rows(self.pool, self.table, lens, i)
            want, w, reach, size = C.attend(self.q[i].double().numpy(), k, v, self.scale, self.G)
            U.check_out(out[i], want, reach, size, self.D, self.scale, p_step, (what, i, n))
            if scores is not None:
                got = scores[i].double().cpu().numpy()
                U.check_scores(got[:, :n], self.before[i, :, :n].astype(float), w, size, self.D, self.scale,
                               (what, i, n))
                assert (got[:, n:] == self.before[i, :, n:]).all()

    def run(self, scores=False, blocks=None, **kw):
        q, pool, table, lens = self.device()
        plan = bd.plan_mx4(bd.mx4_shape(pool, table, q.shape[1]), "cuda", scores=scores, blocks=blocks)
        s = torch.from_numpy(self.before).cuda() if scores else None
        out = bd.mx4_decode(q, pool, table, lens, 16, self.scale, plan=plan, scores=s)
        again = bd.mx4_decode(q, pool, table, lens, 16, self.scale, plan=plan,
                              scores=s.clone() if scores else None)
        torch.cuda.synchronize()
        assert bd.workspace_status(plan) == 0
        assert torch.equal(out, again)
        self.check(out, s, what=(scores, blocks), **kw)


EDGES = [0, 1, 15, 16, 17, 31, 33, 500, 0, 129]


@pytest.mark.parametrize("blocks", [None, 1, 2, 3, 37, 1000])
@pytest.mark.parametrize("G,D", [(4, 128), (1, 64)])
@pytest.mark.parametrize("scores", [False, True])
def test_lengths_and_grids(blocks, G, D, scores):
    Case(EDGES, 2, G, D).run(scores, blocks)


@pytest.mark.parametrize("G", [2, 3, 5, 7, 8, 9, 15, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_group_sizes(G, D):
    c = Case([77, 1, 300], 2, G, D, seed=G)
    c.run(True)
    c.run(False, 5)


@pytest.mark.parametrize("H,lens", [(1, [1]), (1, [9001]), (8, [5000, 3]), (3, [16] * 300), (1, [1] * 4096)])
def test_shapes_of_batches(H, lens):
    Case(lens, H, 1 if len(lens) > 1000 else 4, 64, seed=H).run(len(lens) < 1000)


def test_all_rows_empty():
    c = Case([0, 0], 2, 4, 128)
    q, pool, table, lens = c.device()
    scores = torch.from_numpy(c.before).cuda()
    plan = bd.plan_mx4(bd.mx4_shape(pool, table, 8), "cuda", scores=True)
    out = torch.full_like(q, 3.0)
    bd.mx4_decode(q, pool, table, lens, 16, 1.0, plan=plan, scores=scores, out=out)
    assert (out == 0).all() and (scores.cpu().numpy() == c.before).all()


@pytest.mark.parametrize("spread", [3, 6, 9, 20, 60])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_far_apart(spread, D):
    """V's scales leave the f16 window: bf16 takes the product."""
    for G in (4, 16):
        Case([200, 31, 700], 2, G, D, seed=spread, spread=spread).run(False, p_step=U.BF16_HALF)


@pytest.mark.parametrize("zeros", [0.1, 0.9, 1.0])
def test_blocks_of_zeros(zeros):
    for D in (64, 128):
        c = Case([200, 31, 700], 2, 4, D, zeros=zeros)
        c.run(True, p_step=U.BF16_HALF)


@pytest.mark.parametrize("low,high", [(1, 6), (200, 252), (1, 252)])
def test_values_at_the_ends_of_the_range(low, high):
    """V's scales near the smallest and largest; K's stay ordinary."""
    c = Case([100, 17], 1, 4, 64, seed=low)
    v = c.pool[:, :, 17 * 64 - 32:]
    c.pool[:, :, 17 * 64 - 32:] = np.where(v == 255, 255, c.rng.integers(low, high + 1, v.shape))
    c.run(False, p_step=U.BF16_HALF)


@pytest.mark.parametrize("q_scale", [0.0, 1e-38, 1e-30, 1e30])
def test_queries_of_any_magnitude(q_scale):
    c = Case([100, 17, 40], 2, 4, 128, q_scale=q_scale)
    if q_scale:
        c.scale = c.scale / q_scale if q_scale > 1e-37 else 2.0 ** 100
    c.run(True)


def test_peaked_softmax_over_a_long_row():
    Case([4000], 1, 8, 128, q_scale=30.0).run(True)


@pytest.mark.parametrize("exponent", [18, 19, 21, 60, -100])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scores", [False, True])
def test_logits_whose_floats_are_far_apart(exponent, D, scores):
    """Queries of 1 and -1 on unit scales: products are multiples of 1/2, exact in fp32, so equal ones give equal
    logits and the others lie 2^(exponent - 1) apart, which leaves them no weight.  Logits of 2^27 and more cannot be
    shifted by small amounts."""
    c = Case([1, 40, 700, 3, 16], 2, 4, D, seed=exponent + 200)
    c.pool[:, :, 16 * D:16 * D + D // 2] = np.where(c.pool[:, :, 16 * D:16 * D + D // 2] == 255, 255, 127)
    c.q = c.q.sign()
    c.scale = 2.0 ** exponent
    q, pool, table, lens = c.device()
    for blocks in (None, 3):
        plan = bd.plan_mx4(bd.mx4_shape(pool, table, q.shape[1]), "cuda", scores=scores, blocks=blocks)
        s = torch.from_numpy(c.before).cuda() if scores else None
        out = bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=s).double().cpu().numpy()
        assert bd.workspace_status(plan) == 0
        for i, n in enumerate(c.lens):
            k, v = U.mx4_rows(c.pool, c.table, c.lens, i)
            want, w, reach, size = C.attend(c.q[i].double().numpy(), k, v, c.scale, c.G)
            exact = np.zeros_like(size)  # no error in the logits that count
            U.check_out(out[i], want, reach, exact, D, c.scale, U.F16_HALF, (blocks, i))
            if scores:
                got = s[i].double().cpu().numpy()
                U.check_scores(got[:, :n], c.before[i, :, :n].astype(float), w, exact, D, c.scale, (blocks, i))


def test_infinities_and_nan_stay_in_their_rows():
    c = Case([40, 40, 40], 1, 4, 128)
    D = c.D
    c.pool[c.table[0, 1], 0, 16 * D + 3 * (D // 32)] = 255           # a K scale of row 0
    c.pool[c.table[1, 1], 0, 16 * D + D // 2 + 2 * (D // 32) + 1] = 255  # the V scale of row 1's dims 32 to 63
    c.q[2, 1, 5] = float("inf")
    q, pool, table, lens = c.device()
    plan = bd.plan_mx4(bd.mx4_shape(pool, table, 4), "cuda", scores=True)
    scores = torch.from_numpy(c.before).cuda()
    out = bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=scores).float().cpu()
    assert torch.isnan(out[0]).all() and torch.isnan(scores[0, :, :40]).all()
    assert torch.isnan(out[1, :, 32:64]).all() and torch.isfinite(out[1, :, :32]).all()
    assert torch.isfinite(out[1, :, 64:]).all() and torch.isfinite(scores[1]).all()
    assert torch.isnan(out[2, 1]).all() and torch.isfinite(out[2, [0, 2, 3]]).all()
    assert torch.isnan(scores[2, :, :40]).all() and torch.isfinite(scores[:, :, 40:]).all()


def test_strided_pool():
    c = Case([100, 17, 40], 2, 4, 128)
    q, pool, table, lens = c.device()
    wide = torch.full((pool.shape[0] + 1, 3, pool.shape[2] + 16), 255, dtype=torch.uint8, device="cuda")
    view = wide[1:, 1:, :pool.shape[2]]
    view.copy_(pool)
    out = bd.mx4_decode(q, view, table, lens, 16, c.scale)
    assert torch.equal(out, bd.mx4_decode(q, pool, table, lens, 16, c.scale))
    c.check(out)


def test_replayed_graph_with_lengths_changed_on_the_device():
    c = Case([200, 64, 17], 2, 4, 128, max_pages=13, poison=False)
    q, pool, table, lens = c.device()
    plan = bd.plan_mx4(bd.mx4_shape(pool, table, 8), "cuda", scores=True)
    scores, out = torch.from_numpy(c.before).cuda(), torch.empty_like(q)

    def step(stream=None):
        bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan, scores=scores, out=out, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for now in ([200, 64, 17], [3, 0, 16], [0, 0, 0], [200, 1, 17]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        scores.copy_(torch.from_numpy(c.before))
        g.replay()
        torch.cuda.synchronize()
        assert bd.workspace_status(plan) == 0
        c.check(out, scores, lens=now)


def test_two_calls_at_once_with_plans_of_their_own():
    cases = [Case([3000, 100], 4, 4, 128, seed=s) for s in (1, 2)]
    state = [c.device() for c in cases]
    plans = [bd.plan_mx4(bd.mx4_shape(s[1], s[2], 16), "cuda") for s in state]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [bd.mx4_decode(*s, 16, c.scale, plan=p, stream=st) for c, s, p, st in zip(cases, state, plans, streams)]
    torch.cuda.synchronize()
    for c, out in zip(cases, outs):
        c.check(out)


def test_bad_lengths_and_pages_are_reported():
    c = Case([100, 40], 2, 4, 64)
    q, pool, table, lens = c.device()
    shape = bd.mx4_shape(pool, table, 8)
    plan = bd.plan_mx4(shape, "cuda")
    table[1, 2] = -5
    bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan)
    assert bd.workspace_status(plan) == 4
    plan = bd.plan_mx4(shape, "cuda")
    table.clamp_(0, pool.shape[0] - 1)
    lens[1] = 10**6
    out = bd.mx4_decode(q, pool, table, lens, 16, c.scale, plan=plan)
    assert bd.workspace_status(plan) == 2
    c.check(out[:1], lens=[100])


# ---------------------------------------------------------------------------
# the operators together

def test_prompt_steps_and_eviction_together():
    """A prompt goes into the 4-bit cache, steps append a token and attend with scores, an eviction shrinks the
    cache, and the next steps run on what is left; the oracle follows each stage from the GPU's own cache bytes."""
    rng = np.random.default_rng(11)
    H, G, D, prompt, budget, recent = 2, 4, 128, [70, 33, 50], 48, 8
    B, max_pages = 3, 6
    table = torch.from_numpy(rng.permutation(B * max_pages).reshape(B, max_pages).astype(np.int32)).cuda()
    pool = bd.mx4_pool(B * max_pages, H, D, "cuda")
    plan = bd.plan_mx4(bd.mx4_shape(pool, table, H * G), "cuda", scores=True)
    evict = bd.plan_evict(B, H, max_pages, "cuda")
    scores = torch.zeros(B, H, max_pages * 16, device="cuda")
    positions = torch.zeros(B, H, max_pages * 16, dtype=torch.int32, device="cuda")
    for i, n in enumerate(prompt):
        positions[i, :, :n] = torch.arange(n, dtype=torch.int32)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    indptr = torch.tensor([0, 70, 103, 153], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(153, H, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    bd.mx4_append(k, v, pool, table, lens, plan=plan, indptr=indptr)
    lens += torch.tensor(prompt, dtype=torch.int32, device="cuda")
    scale, at = D ** -0.5, list(prompt)
    total = np.zeros((B, H, max_pages * 16))
    for step in range(4):
        k, v = (torch.randn(B, H, D, device="cuda").to(torch.bfloat16) for _ in range(2))
        bd.mx4_append(k, v, pool, table, lens, plan=plan)
        for i, n in enumerate(lens.tolist()):
            positions[i, :, n] = at[i]
            at[i] += 1
        lens += 1
        q = torch.randn(B, H * G, D, device="cuda").to(torch.bfloat16)
        out = bd.mx4_decode(q, pool, table, lens, 16, scale, plan=plan, scores=scores).double().cpu().numpy()
        now, host = lens.tolist(), pool.cpu().numpy()
        for i, n in enumerate(now):
            rows = U.mx4_rows(host, table.cpu().numpy(), now, i)
            want, w, reach, size = C.attend(q[i].double().cpu().numpy(), *rows, scale, G)
            U.check_out(out[i], want, reach, size, D, scale, U.BF16_HALF, (step, i))
            U.check_scores(scores[i].double().cpu().numpy()[:, :n], total[i, :, :n], w, size, D, scale, (step, i))
        total = scores.double().cpu().numpy()
        if step == 1:
            planes = [p.cpu().numpy() for p in bd.mx4_planes(pool)]
            want = C.evict(scores.cpu().numpy(), positions.cpu().numpy(), planes, table.cpu().numpy(), now, budget,
                           recent)
            lens = bd.evict_tokens(scores, bd.mx4_planes(pool), table, lens, budget, recent, positions=positions,
                                   plan=evict)
            assert lens.tolist() == want[3] == [48, 35, 48]
            assert (scores.cpu().numpy() == want[0]).all() and (positions.cpu().numpy() == want[1]).all()
            for p, x in zip(bd.mx4_planes(pool), want[2]):
                assert (p.cpu().numpy() == x).all()
            # the newest tokens are still the last ones
            assert positions[0, 0, 40:48].tolist() == list(range(64, 72))
            total = scores.double().cpu().numpy()
    assert bd.workspace_status(plan) == 0 and bd.workspace_status(evict) == 0


def test_refusals():
    c = Case([100, 40], 2, 4, 64)
    q, pool, table, lens = c.device()
    plan = bd.plan_mx4(bd.mx4_shape(pool, table, 8), "cuda")
    scored = bd.plan_mx4(bd.mx4_shape(pool, table, 8), "cuda", scores=True)
    scores = torch.from_numpy(c.before).cuda()

    def decode(q=q, pool=pool, table=table, lens=lens, **kw):
        return bd.mx4_decode(q, pool, table, lens, 16, 1.0, **{"plan": plan, **kw})

    for kw in (dict(q=q[:1]), dict(q=q[:, :4]), dict(q=q.cpu()), dict(pool=pool[:, :1]), dict(pool=pool[:-1]),
               dict(pool=pool[..., :-1]), dict(table=table[:1]), dict(lens=lens[:1]), dict(scores=scores),
               dict(plan=scored), dict(plan=scored, scores=scores[:, :, :9]), dict(out=q[:1]),
               dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            decode(**kw)
    for kw in (dict(q=q.half()), dict(pool=pool.char()), dict(table=table.long()), dict(out=q.float())):
        with pytest.raises(TypeError):
            decode(**kw)
    with pytest.raises(bd.PkvError):
        bd.mx4_decode(q, pool, table, lens, 32, 1.0, plan=plan)
    with pytest.raises(bd.PkvError):
        bd.plan_mx4(bd.mx4_shape(pool, table, 8), "cuda", blocks=4000)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    ind = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")

    def append(k=k, v=k, **kw):
        return bd.mx4_append(k, v, pool, table, lens, plan=plan, **kw)

    for kw in (dict(k=k[:1]), dict(k=k[:1], v=k[:1]), dict(k=k[..., :32]), dict(k=k[:, :1]), dict(indptr=ind[:2]),
               dict(k=k.cpu()), dict(k=k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            append(**kw)
    for kw in (dict(k=k.float()), dict(indptr=ind.long())):
        with pytest.raises(TypeError):
            append(**kw)
    odd = torch.zeros(2, 2, 65, dtype=torch.bfloat16, device="cuda")[..., :64]
    with pytest.raises(bd.PkvError):
        append(k=odd, v=odd)
    with pytest.raises(ValueError):
        bd.mx4_read(pool, table, lens, 3, plan=plan)
    with pytest.raises(ValueError):
        bd.mx4_pool(4, 2, 96, "cuda")
