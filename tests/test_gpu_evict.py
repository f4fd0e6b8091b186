"""Eviction by accumulated attention weight (evict_tokens) against the oracle, bit for bit: budgets and windows at their
limits, scores with ties, NaN and infinities, planes of every copy width, layouts, strides, graphs, bad pages."""
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


def make_scores(rng, kind, B, H, T):
    if kind == "equal":
        return np.full((B, H, T), 0.25, np.float32)
    if kind == "few":  # many ties
        return rng.integers(0, 3, (B, H, T)).astype(np.float32)
    if kind == "odd":  # both zeros, negatives, subnormals, infinities, NaN
        pick = np.array([0.0, -0.0, 1e-42, -1e-42, np.inf, -np.inf, np.nan, -np.nan, 1.5, -1.5], np.float32)
        return pick[rng.integers(0, len(pick), (B, H, T))]
    if kind == "rising":
        return np.broadcast_to(np.arange(T, dtype=np.float32), (B, H, T)).copy()
    return rng.exponential(1.0, (B, H, T)).astype(np.float32)


class Case:
    def __init__(self, lens, H, widths=(8,), kind="exp", seed=1, dtype=np.uint8, max_pages=None):
        rng = np.random.default_rng(seed)
        self.lens, self.H = lens, H
        self.max_pages = max_pages or max(1, max(-(-n // 16) for n in lens))
        self.table, self.pages = U.scattered_table(rng, lens, self.max_pages)
        T = self.max_pages * 16
        self.scores = make_scores(rng, kind, len(lens), H, T)
        self.positions = rng.integers(-2**31, 2**31, (len(lens), H, T)).astype(np.int32)
        self.planes = [rng.integers(0, 256, (self.pages, H, 16, w)).astype(dtype) for w in widths]

    def device(self):
        return (torch.from_numpy(self.scores).cuda(), torch.from_numpy(self.positions).cuda(),
                [torch.from_numpy(p).cuda() for p in self.planes], torch.from_numpy(self.table).cuda(),
                torch.tensor(self.lens, dtype=torch.int32, device="cuda"))

    def want(self, budget, recent):
        return C.evict(self.scores, self.positions, self.planes, self.table, self.lens, budget, recent)

    def check(self, got, budget, recent, what=""):
        scores, positions, planes, lens = got
        ws, wp, wpl, wl = self.want(budget, recent)
        assert lens.tolist() == wl, what
        assert (positions.cpu().numpy() == wp).all(), what
        assert (scores.cpu().numpy().view(np.int32) == ws.view(np.int32)).all(), what
        for p, w in zip(planes, wpl):
            assert (p.cpu().numpy() == w).all(), what

    def run(self, budget, recent, **kw):
        scores, positions, planes, table, lens = self.device()
        plan = bd.plan_evict(len(self.lens), self.H, self.max_pages, "cuda")
        new = bd.evict_tokens(scores, planes, table, lens, budget, recent, positions=positions, plan=plan, **kw)
        torch.cuda.synchronize()
        assert bd.workspace_status(plan) == 0
        assert lens.tolist() == self.lens
        self.check((scores, positions, planes, new), budget, recent, (budget, recent, kw))


@pytest.mark.parametrize("kind", ["exp", "equal", "few", "odd", "rising"])
@pytest.mark.parametrize("budget,recent", [(0, 0), (1, 0), (1, 1), (5, 2), (16, 16), (17, 0), (100, 30), (100, 99),
                                           (511, 128), (512, 0), (600, 1)])
def test_budgets_windows_and_scores(kind, budget, recent):
    Case([0, 1, 5, 16, 17, 33, 100, 101, 513, 600], 2, (8, 16), kind).run(budget, recent)


@pytest.mark.parametrize("n", [2, 31, 1000, 1024, 1025, 4097])
def test_one_row_one_head(n):
    for kind in ("exp", "odd"):
        c = Case([n], 1, (4,), kind, seed=n)
        for budget, recent in ((n - 1, 0), (n - 1, min(7, n - 1)), (n // 2, n // 4), (1, 0)):
            c.run(budget, recent)


def test_many_pairs():
    lens = [int(x) for x in np.random.default_rng(7).integers(0, 200, 70)]
    Case(lens, 8, (16, 2)).run(64, 16)


def test_a_row_past_the_keys_a_block_holds():
    # eight blocks of 16384 keys hold 131072 tokens; the rest is read again
    c = Case([140003], 1, (1,), "few")
    c.run(70000, 5000)
    c.run(139999, 137000)


@pytest.mark.parametrize("width,dtype", [(1, np.uint8), (2, np.uint8), (3, np.uint8), (4, np.uint8), (6, np.uint8),
                                         (24, np.uint8), (64, np.float16), (5, np.int32), (3, np.float64),
                                         (128, np.float32)])
def test_planes_of_every_copy_width(width, dtype):
    Case([100, 40], 2, (width, 16), dtype=dtype, seed=width).run(33, 8)


def test_eight_planes():
    Case([100, 40], 2, (1, 2, 4, 8, 16, 32, 64, 3)).run(33, 8)


def test_nhd_layout_and_views_of_a_combined_cache():
    c = Case([100, 40, 7], 2, (64, 64))
    budget, recent = 20, 5
    want = c.want(budget, recent)
    # K and V as the halves of one [pages][2][16][H][X] cache, rows padded behind X
    kv = torch.full((c.pages, 2, 16, 2, 64 + 16), 99, dtype=torch.uint8, device="cuda")
    for i, p in enumerate(c.planes):
        kv[:, i, :, :, :64] = torch.from_numpy(p).cuda().transpose(1, 2)
    scores, positions, _, table, lens = c.device()
    store = torch.full((3, 2, 3, scores.shape[2] + 3), 7.0, device="cuda")
    view = store[:, :, 1, 2:2 + scores.shape[2]]
    view.copy_(scores)
    new = bd.evict_tokens(view, (kv[:, 0, :, :, :64], kv[:, 1, :, :, :64]), table, lens, budget, recent,
                          positions=positions, layout="NHD")
    planes = [kv[:, i, :, :, :64].transpose(1, 2).contiguous() for i in range(2)]
    c.check((view, positions, planes, new), budget, recent)
    assert (kv[..., 64:] == 99).all()
    view.fill_(7.0)
    assert (store == 7.0).all()
    assert want[3] == new.tolist()


def test_without_positions_and_on_another_stream():
    c = Case([100, 40], 2, (16,))
    scores, _, planes, table, lens = c.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.full((5,), -1, dtype=torch.int32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    got = bd.evict_tokens(scores, planes, table, lens, 33, 8, stream=side, out=out)
    side.synchronize()
    assert got.tolist() == [33, 33, -1, -1, -1]
    ws, _, wpl, _ = c.want(33, 8)
    assert (scores.cpu().numpy() == ws).all() and (planes[0].cpu().numpy() == wpl[0]).all()


def test_replayed_graph_with_lengths_changed_on_the_device():
    c = Case([100, 90, 33], 2, (16,))
    scores, positions, planes, table, lens = c.device()
    plan = bd.plan_evict(3, 2, c.max_pages, "cuda")
    out = torch.empty(3, dtype=torch.int32, device="cuda")
    saved = [t.clone() for t in (scores, positions, planes[0])]
    bd.evict_tokens(scores, planes, table, lens, 20, 4, positions=positions, plan=plan, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bd.evict_tokens(scores, planes, table, lens, 20, 4, positions=positions, plan=plan, out=out)
    for now in ([100, 90, 33], [20, 21, 0], [99, 3, 32]):
        for t, s in zip((scores, positions, planes[0]), saved):
            t.copy_(s)
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        full, c.lens = c.lens, now
        c.check((scores, positions, planes, out), 20, 4, now)
        c.lens = full


def test_two_calls_at_once_with_plans_of_their_own():
    cases = [Case([3000, 100], 4, (64,), seed=s) for s in (1, 2)]
    state = [c.device() for c in cases]
    plans = [bd.plan_evict(2, 4, c.max_pages, "cuda") for c in cases]
    outs = [torch.empty(2, dtype=torch.int32, device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for (scores, positions, planes, table, lens), plan, out, st in zip(state, plans, outs, streams):
        bd.evict_tokens(scores, planes, table, lens, 700, 64, positions=positions, plan=plan, out=out, stream=st)
    torch.cuda.synchronize()
    for c, (scores, positions, planes, _, _), out in zip(cases, state, outs):
        c.check((scores, positions, planes, out), 700, 64)


def test_bad_lengths_and_pages_are_reported():
    c = Case([100, 90, 33], 2, (16,))
    scores, positions, planes, table, lens = c.device()
    plan = bd.plan_evict(3, 2, c.max_pages, "cuda")
    lens.copy_(torch.tensor([-3, 100000, 33], dtype=torch.int32))
    before = [t.clone() for t in (scores, positions, planes[0])]
    new = bd.evict_tokens(scores, planes, table, lens, 40, 4, positions=positions, plan=plan)
    assert bd.workspace_status(plan) == 2
    assert new.tolist() == [0, c.max_pages * 16, 33]
    for t, b in zip((scores, positions, planes[0]), before):
        assert torch.equal(t, b)
    # a page id out of range: its tokens are not moved, the other rows are as ever
    lens.copy_(torch.tensor([100, 90, 33], dtype=torch.int32))
    table[1, 2] = 10**6
    plan = bd.plan_evict(3, 2, c.max_pages, "cuda")
    new = bd.evict_tokens(scores, planes, table, lens, 20, 4, positions=positions, plan=plan)
    assert bd.workspace_status(plan) == 4
    ws, wp, wpl, wl = c.want(20, 4)
    assert new.tolist() == wl
    for i in (0, 2):
        assert (scores[i].cpu().numpy() == ws[i]).all()
        for t in range(20):
            at = c.table[i, t // 16]
            assert (planes[0][at, :, t % 16].cpu().numpy() == wpl[0][at, :, t % 16]).all()


def test_refusals():
    c = Case([100, 40], 2, (16,))
    scores, positions, planes, table, lens = c.device()

    def call(s=scores, p=planes, b=20, r=4, **kw):
        return bd.evict_tokens(s, p, table, lens, b, r, **kw)

    for kw in (dict(r=-1), dict(r=21), dict(b=-1), dict(b=2**31), dict(p=[]), dict(p=planes * 9),
               dict(p=[planes[0][:, :1]]), dict(p=[planes[0][:, :, :8]]), dict(p=[planes[0].transpose(2, 3)]),
               dict(p=[planes[0].cpu()]), dict(p=[planes[0][:, :, :1].expand(-1, -1, 16, -1)]),
               dict(p=[planes[0], planes[0][:1]]), dict(s=scores[:, :, :50]), dict(s=scores[:1]),
               dict(s=scores[:1].expand(2, -1, -1)), dict(positions=positions[:, :, :50]), dict(out=lens),
               dict(out=torch.zeros(1, dtype=torch.int32, device="cuda")), dict(layout="DHN"),
               dict(plan=bd.plan_evict(3, 2, c.max_pages, "cuda")), dict(layout="NHD")):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(s=scores.double()), dict(positions=positions.long()), dict(out=lens.long())):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(bd.PkvError):
        call(p=[torch.zeros(c.pages, 2, 16, 5000, dtype=torch.uint8, device="cuda")])
