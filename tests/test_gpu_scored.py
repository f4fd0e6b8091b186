"""Decode that accumulates attention weights (paged_decode_scored) against the fp64 oracle: every plan it takes,
lengths around page borders, group sizes, strided scores, replayed graphs with other lengths, other streams."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from paged_kv_gqa_17_b200 import binding as bd

from . import cache_util as U

pytestmark = pytest.mark.gpu

ANY = (0, 2**31 - 1, 0, 2**31 - 1)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_gqa_17_b200 import build

    build.build()
    bd.lib()


def rule(mode, S=1, Cp=0, flags=0):
    return [bd.Rule(*ANY, mode, S, Cp, flags)]


class Case:
    """A batch with NaN in every slot no row owns, scores with room and a sentinel past every row's end."""

    def __init__(self, lens, H_kv, G, D, layout="HND", seed=1, max_pages=None, room=5, q_scale=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.H_kv, self.G, self.D, self.layout = lens, H_kv, G, D, layout
        self.max_pages = max_pages or max(1, max(-(-n // 16) for n in lens))
        self.table, pages = U.scattered_table(rng, lens, self.max_pages)
        self.scale = D ** -0.5
        kv = torch.from_numpy(rng.standard_normal((2, pages, H_kv, 16, D))).to(torch.bfloat16)
        live = torch.zeros(pages, 16, dtype=torch.bool)
        for i, n in enumerate(lens):
            for t in range(n):
                live[self.table[i, t // 16], t % 16] = True
        kv[(~live)[None, :, None, :, None].expand_as(kv)] = float("nan")
        self.k, self.v = kv
        self.q = torch.from_numpy(rng.standard_normal((len(lens), H_kv * G, D)) * q_scale).to(torch.bfloat16)
        self.before = rng.random((len(lens), H_kv, self.max_pages * 16 + room)).astype(np.float32)
        k, v = (x if layout == "HND" else x.transpose(1, 2).contiguous() for x in (self.k, self.v))
        self.kd, self.vd, self.qd = k.cuda(), v.cuda(), self.q.cuda()
        self.td = torch.from_numpy(self.table).cuda()
        self.ld = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def shape(self):
        return bd.shape_of(self.qd, self.kd, self.td, self.layout, self.vd)

    def rows(self, x, i):
        n = self.lens[i]
        pages = self.table[i, :-(-n // 16)]
        return x[torch.from_numpy(pages).long()].double().numpy().transpose(1, 0, 2, 3).reshape(
            self.H_kv, -1, self.D)[:, :n]

    def check(self, out, scores, times=1, lens=None, what=""):
        out, scores = out.double().cpu().numpy(), scores.double().cpu().numpy()
        full = self.lens
        self.lens = lens or full
        for i, n in enumerate(self.lens):
            want, w, reach, size = C.attend(self.q[i].double().numpy(), self.rows(self.k, i), self.rows(self.v, i),
                                            self.scale, self.G)
            U.check_out(out[i], want, reach, size, self.D, self.scale, U.BF16_HALF, (what, i, n))
            before = self.before[i].astype(np.float64)
            for _ in range(times):
                U.check_scores(scores[i, :, :n], before[:, :n] + (times - 1) * w, w, size * times, self.D, self.scale,
                               (what, i, n))
                break
            assert (scores[i, :, n:] == before[:, n:]).all(), (what, i, n, "past the end")
        self.lens = full

    def run(self, plan, **kw):
        scores = torch.from_numpy(self.before).cuda()
        out = bd.paged_decode_scored(self.qd, self.kd, self.vd, self.td, self.ld, 16, self.scale, scores, plan=plan,
                                     layout=self.layout, **kw)
        torch.cuda.synchronize()
        assert bd.workspace_status(plan) == 0
        return out, scores


EDGES = [0, 1, 15, 16, 17, 31, 33, 500]
PLANS = [("policy", None, {}), ("no split", rule(0), {}), ("split 1", rule(1, 1), {}), ("split 4", rule(1, 4), {}),
         ("split 40", rule(1, 40), {}), ("split deep", rule(1, 3, 0, 4), {}), ("queue 1", rule(2, 1, 1), {}),
         ("queue 5", rule(2, 1, 5), {}), ("queue merge kernel", rule(2, 1, 2, 1), {}), ("split merge kernel", rule(1, 7, 0, 1), {}),
         ("queue no pdl", rule(2, 1, 3, 2), {}), ("queue early", rule(2, 1, 3, 16), {}),
         ("device fill", rule(2, 296, 0), {"device_queue": True}),
         ("device fill deep", rule(2, 20, 0, 4), {"device_queue": True, "fill_blocks": 20}),
         ("device builder", rule(2, 296, 0), {"device_queue": True, "device_fill": False})]


@pytest.mark.parametrize("what,rules,kw", PLANS, ids=[p[0] for p in PLANS])
@pytest.mark.parametrize("G,D", [(4, 128), (1, 64)])
def test_every_plan(what, rules, kw, G, D):
    c = Case(EDGES, 2, G, D)
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", rules=rules, scores=True, **kw)
    out, scores = c.run(plan)
    c.check(out, scores, what=what)
    # the output has the bits of the decode without scores, and a second call adds the same weights again
    plain = bd.plan_decode(c.lens, c.shape(), "cuda", rules=rules, **kw)
    if plain.plan.tuple()[:3] == plan.plan.tuple()[:3] and not plain.plan.flags & bd.FLAG_CLUSTER_MERGE:
        assert torch.equal(out, bd.paged_decode(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, plan=plain))
    again = scores.clone()
    bd.paged_decode_scored(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, again, plan=plan)
    c.check(out, again, times=2, what=what)


@pytest.mark.parametrize("G", [2, 3, 7, 8, 9, 16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_group_sizes_and_layouts(G, D, layout):
    c = Case([77, 1, 300], 2, G, D, layout, seed=G, q_scale=3.0)
    for rules in (rule(0), rule(1, 3), rule(2, 1, 4)):
        plan = bd.plan_decode(c.lens, c.shape(), "cuda", rules=rules, scores=True)
        c.check(*c.run(plan), what=(G, D, rules[0].tuple()))


def test_a_long_row_and_the_built_in_policy():
    c = Case([9000, 2000], 8, 4, 128, seed=9)
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", scores=True)
    c.check(*c.run(plan))


def test_scores_as_a_view():
    c = Case([40, 100], 2, 4, 64, seed=3)
    T = c.before.shape[2]
    store = torch.full((2, 3, 2, T + 7), -5.0, device="cuda")
    view = store[:, 1, :, 3:3 + T]
    view.copy_(torch.from_numpy(c.before))
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", scores=True)
    out = bd.paged_decode_scored(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, view, plan=plan)
    c.check(out, view)
    store[:, 1, :, 3:3 + T] = -5.0
    assert (store == -5.0).all()


def test_no_plan_and_another_stream():
    c = Case(EDGES, 2, 4, 128, seed=4)
    scores = torch.from_numpy(c.before).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = bd.paged_decode_scored(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, scores, stream=side)
    side.synchronize()
    c.check(out, scores)


def test_replayed_graph_with_lengths_changed_on_the_device():
    c = Case([200, 64, 17], 2, 4, 128, seed=5, max_pages=13)
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", rules=rule(2, 296, 0), scores=True, device_queue=True)
    scores = torch.zeros(c.before.shape, device="cuda")
    out = torch.empty_like(c.qd)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        bd.paged_decode_scored(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, scores, plan=plan, out=out)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bd.paged_decode_scored(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, scores, plan=plan, out=out)
    for lens in ([200, 64, 17], [3, 0, 16], [200, 1, 17]):
        c.ld.copy_(torch.tensor(lens, dtype=torch.int32))
        scores.copy_(torch.from_numpy(c.before))
        g.replay()
        torch.cuda.synchronize()
        assert bd.workspace_status(plan) == 0
        # a shorter row's tail slots were tokens: the check reads only the first lens[i]
        c.check(out, scores, lens=lens)


def test_a_row_whose_logits_are_all_minus_infinity_gets_no_weight():
    c = Case([20, 20], 1, 2, 64, seed=6)
    c.k[torch.from_numpy(c.table[0, :2]).long()] = -3.0e38
    c.q[0] = 3.0e38  # products overflow to -inf
    c.kd.copy_(c.k)
    c.qd.copy_(c.q)
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", scores=True)
    out, scores = c.run(plan)
    assert (out[0] == 0).all()
    assert (scores[0].cpu().numpy() == c.before[0]).all()
    assert torch.isfinite(scores).all()


def test_nan_in_a_key_shows_in_its_row_only():
    c = Case([20, 20], 1, 2, 64, seed=6)
    c.k[c.table[0, 0], 0, 3] = float("nan")
    c.kd.copy_(c.k)
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", scores=True)
    out, scores = c.run(plan)
    assert torch.isnan(out[0]).all() and torch.isnan(scores[0, :, :20]).all()
    assert torch.isfinite(out[1]).all() and torch.isfinite(scores[1]).all()
    assert (scores[0, :, 20:].cpu().numpy() == c.before[0, :, 20:]).all()


def test_device_errors_are_reported():
    c = Case([40, 100], 2, 4, 64, seed=3)
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", scores=True)
    c.ld.copy_(torch.tensor([40, 1 << 20], dtype=torch.int32))
    scores = torch.zeros(c.before.shape, device="cuda")
    c.td[1] = c.td[0, 0]  # pages for the clamped length
    plan = bd.plan_decode([112, 112], c.shape(), "cuda", rules=rule(1, 2), scores=True)
    bd.paged_decode_scored(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, scores, plan=plan)
    assert bd.workspace_status(plan) == 2


def test_refusals():
    c = Case([40, 100], 2, 4, 64, seed=3)
    scores = torch.from_numpy(c.before).cuda()
    plain = bd.plan_decode(c.lens, c.shape(), "cuda")
    plan = bd.plan_decode(c.lens, c.shape(), "cuda", scores=True)

    def call(s=scores, p=plan, **kw):
        return bd.paged_decode_scored(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, s, plan=p, **kw)

    for bad in (scores[:1], scores[:, :1], scores[:, :, :100], scores.transpose(1, 2),
                scores[:1].expand(2, -1, -1), scores.cpu(), scores[0]):
        with pytest.raises(ValueError):
            call(bad)
    with pytest.raises(TypeError):
        call(scores.double())
    with pytest.raises(ValueError):
        call(p=plain)
    with pytest.raises(bd.PkvError):
        bd.paged_decode(c.qd, c.kd, c.vd, c.td, c.ld, 16, c.scale, plan=plan)
    with pytest.raises(ValueError):
        bd.plan_decode(c.lens, c.shape(), "cuda", scores=True, shared_prefix_table=c.table)
    with pytest.raises(ValueError):
        bd.plan_decode(c.lens, c.shape(), "cuda", plan=bd.Plan(3, 4, 0, 0), scores=True)
