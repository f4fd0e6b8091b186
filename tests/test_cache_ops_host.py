"""The cache operators on the CPU: workspace sizes, and refusals of the C entry points, which come before any CUDA
call, and of the binding."""
import ctypes

import pytest
import torch

from paged_kv_gqa_17_b200 import binding as bd

INVALID, UNSUPPORTED, CAPACITY = -1, -2, -3
P = 256  # any aligned non-null address: these calls return before they use it


@pytest.fixture(scope="module")
def L():
    from paged_kv_gqa_17_b200 import build

    build.build()
    return bd.lib()


def shape(B=2, H_q=8, H_kv=2, D=128, P=16, max_pages=4, pages=9):
    return bd.make_shape(B, H_q, H_kv, D, P, max_pages, pages)


def mx4(B=2, H_q=8, H_kv=2, D=128, P=16, max_pages=4, pages=9, page=None, head=None):
    return bd.Shape(B, H_q, H_kv, D, P, max_pages, pages, 0, page or 17 * D * H_kv, head or 17 * D, D // 2)


def test_a_scored_plan_holds_the_logits_and_every_state(L):
    s = shape(3, 20, 4, 64, 16, 10, 40)  # G = 5, logits laid out for 8 heads
    logits = 3 * 4 * 160 * 8 * 4
    for plan in (bd.Plan(0, 1, 0, 0), bd.Plan(1, 4, 3, 0), bd.Plan(2, 4, 3, 0)):
        scored = bd.Plan(plan.mode, plan.num_splits, plan.chunk_pages, bd.FLAG_SCORES)
        more = bd.workspace_bytes(s, scored, 20) - bd.workspace_bytes(s, plan, 20)
        assert logits <= more <= logits + 3 * 4 * 16 + 12 * 5 * (64 + 2) * 4 + 2048
    lens = [100, 0, 7]
    plain, scored = (bd.plan_counters(lens, s, bd.Plan(1, 4, 3, f)) for f in (0, bd.FLAG_SCORES))
    assert scored.pop("launches") == plain.pop("launches") + 1 and plain == scored


def test_plan_decode_with_scores_keeps_to_what_the_call_takes(L):
    s = shape(1, 8, 2, 128, 16, 32, 64)
    cluster = [bd.Rule(0, 9, 0, 10**6, 1, 8, 0, 8 | 4)]
    assert bd.plan_decode([500], s, "cpu", rules=cluster, scores=True).plan.tuple() == (1, 8, 4, 4 | 128)
    balanced = [bd.Rule(0, 9, 0, 10**6, 3, 16, 0, 0)]
    plan = bd.plan_decode([500], s, "cpu", rules=balanced, scores=True)
    assert plan.plan.mode == bd.WORK_QUEUE and plan.plan.flags == bd.FLAG_SCORES and plan.n_items <= 16
    device = bd.plan_decode([500], s, "cpu", rules=balanced, scores=True, device_queue=True)
    assert device.plan.flags == bd.FLAG_SCORES | bd.FLAG_DEVICE_FILL
    with pytest.raises(ValueError):
        bd.plan_decode([500], s, "cpu", plan=bd.Plan(3, 16, 0, 0), scores=True)
    with pytest.raises(ValueError):
        bd.plan_decode([500], s, "cpu", scores=True, shared_prefix_table=torch.zeros(1, 32, dtype=torch.int32))


def scored(L, s, plan, scores=P, flags=bd.FLAG_SCORES, fn="pkv_paged_decode_scored", ws_bytes=1 << 30):
    plan = bd.Plan(plan[0], plan[1], plan[2], flags)
    return getattr(L, fn)(P, P, P, P, P, s.page_size, 1.0, P, scores, 64, 32, ctypes.byref(s), ctypes.byref(plan), P, P, 64,
                          P, ws_bytes, None)


def test_scored_decode_refusals(L):
    assert scored(L, shape(), (0, 1, 0), flags=0) == UNSUPPORTED        # a plan without the flag
    assert scored(L, shape(), (3, 4, 0)) == UNSUPPORTED                 # BALANCED
    assert scored(L, shape(), (1, 4, 1), flags=128 | 8) == UNSUPPORTED  # cluster merge
    assert scored(L, shape(), (2, 4, 1), flags=128 | 64) == UNSUPPORTED # prefix-sharing queue
    assert scored(L, shape(), (0, 1, 0), scores=None) == INVALID
    assert scored(L, shape(), (0, 1, 0), scores=2) == UNSUPPORTED       # misaligned
    assert scored(L, shape(), (0, 1, 0), ws_bytes=100) == CAPACITY
    assert scored(L, shape(D=96), (0, 1, 0)) == UNSUPPORTED
    plan, s = bd.Plan(0, 1, 0, bd.FLAG_SCORES), shape()                 # and the flag without scores
    assert L.pkv_paged_decode(P, P, P, P, P, 16, 1.0, P, ctypes.byref(s), ctypes.byref(plan), None, None, 0, P, 1 << 30,
                              None) == UNSUPPORTED


def evict(L, s=None, budget=4, recent=2, planes=1, row_bytes=256, stride=256, scores=P, lens=P, new=2 * P, ws=1 << 30,
          base=P, n=None):
    s = s or shape()
    arr = (bd.Plane * max(1, planes))(*[bd.Plane(base, 16 * stride, 16 * stride, stride, row_bytes, 0)] * planes)
    return L.pkv_evict_tokens(scores, 64, 32, None, 0, 0, arr, planes if n is None else n, P, lens, budget, recent, new,
                              ctypes.byref(s), P, ws, None)


def test_evict_refusals(L):
    assert evict(L, budget=-1, recent=-1) == INVALID
    assert evict(L, recent=5) == INVALID
    assert evict(L, recent=-1) == INVALID
    assert evict(L, n=-1) == INVALID
    assert evict(L, planes=9) == UNSUPPORTED
    assert evict(L, row_bytes=0) == INVALID
    assert evict(L, row_bytes=4097) == UNSUPPORTED
    assert evict(L, stride=-16) == INVALID
    assert evict(L, base=None) == INVALID
    assert evict(L, scores=None) == INVALID
    assert evict(L, new=P) == INVALID                    # the lengths themselves
    assert evict(L, scores=2) == UNSUPPORTED
    assert evict(L, s=shape(P=32)) == UNSUPPORTED
    assert evict(L, s=shape(max_pages=0)) == INVALID
    assert evict(L, s=shape(max_pages=2**26)) == UNSUPPORTED
    assert evict(L, ws=100) == CAPACITY
    assert evict(L, s=shape(B=0)) == 0                   # nothing to do


def decode(L, s=None, blocks=4, flags=0, scores=None, mode=3, chunk=0, page_size=16, q=P, ws=1 << 30, pool=P):
    s, plan = s or mx4(), bd.Plan(mode, blocks, chunk, flags)
    return L.pkv_mx4_decode(q, pool, P, P, page_size, 1.0, P, scores, 64, 32, ctypes.byref(s), ctypes.byref(plan), P, ws, None)


def test_mx4_decode_refusals(L):
    assert decode(L, page_size=32) == INVALID
    assert decode(L, mode=1) == INVALID
    assert decode(L, blocks=0) == INVALID
    assert decode(L, blocks=1025) == UNSUPPORTED
    assert decode(L, flags=bd.FLAG_DEEP_RING) == UNSUPPORTED
    assert decode(L, flags=bd.FLAG_SCORES) == UNSUPPORTED        # the flag without scores
    assert decode(L, scores=P) == UNSUPPORTED                    # scores without the flag
    assert decode(L, s=mx4(H_q=34, H_kv=2)) == UNSUPPORTED       # G = 17
    assert decode(L, s=mx4(H_q=9, H_kv=2)) == INVALID
    assert decode(L, s=mx4(D=96)) == UNSUPPORTED
    assert decode(L, s=mx4(B=4097)) == UNSUPPORTED
    assert decode(L, s=mx4(page=17 * 256 + 8)) == UNSUPPORTED    # records off 16 bytes
    assert decode(L, s=mx4(head=17 * 128 + 4)) == UNSUPPORTED
    assert decode(L, s=mx4(B=4096, H_kv=8, max_pages=2**16)) == UNSUPPORTED  # 2^31 pages
    assert decode(L, pool=P + 8) == UNSUPPORTED
    assert decode(L, q=None) == INVALID
    assert decode(L, ws=100) == CAPACITY
    assert decode(L, s=mx4(B=0)) == 0
    n = ctypes.c_size_t(0)
    s, plan = mx4(), bd.Plan(3, 4, 0, 0)
    assert L.pkv_mx4_workspace_bytes(ctypes.byref(s), ctypes.byref(plan), ctypes.byref(n)) == 0 and n.value % 256 == 0
    assert L.pkv_mx4_workspace_bytes(ctypes.byref(s), None, ctypes.byref(n)) == INVALID


def append(L, s=None, n=2, k=P, stride=128, pool=P, indptr=P):
    s = s or mx4()
    return L.pkv_mx4_append(k, P, stride, 128, 256, 128, pool, P, P, indptr, n, ctypes.byref(s), P, None)


def test_mx4_token_refusals(L):
    assert append(L, n=-1) == INVALID
    assert append(L, n=0) == 0
    assert append(L, k=None) == INVALID
    assert append(L, k=P + 2) == UNSUPPORTED
    assert append(L, stride=132) == UNSUPPORTED
    assert append(L, stride=-128) == UNSUPPORTED
    assert append(L, pool=None) == INVALID
    assert append(L, pool=P + 4) == UNSUPPORTED
    assert append(L, n=3, indptr=None) == INVALID       # one token per row of two
    assert append(L, s=mx4(B=0)) == INVALID
    assert append(L, s=mx4(P=8)) == UNSUPPORTED
    assert append(L, n=2**30) == UNSUPPORTED
    s = mx4()
    assert L.pkv_mx4_read(P, P, P, P, 2, None, P, ctypes.byref(s), P, None) == INVALID
    assert L.pkv_mx4_read(P, P, P, P, 2, P + 2, P, ctypes.byref(s), P, None) == UNSUPPORTED


def test_binding_wants_cuda_tensors_and_whole_records():
    pool = torch.zeros(4, 2, 17 * 64, dtype=torch.uint8)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    scores = torch.zeros(2, 2, 32)
    with pytest.raises(ValueError):
        bd.mx4_decode(q, pool, table, lens, 16, 1.0)
    with pytest.raises(ValueError):
        bd.mx4_append(kv, kv, pool, table, lens)
    with pytest.raises(ValueError):
        bd.mx4_read(pool, table, lens, 2)
    with pytest.raises(ValueError):
        bd.evict_tokens(scores, bd.mx4_planes(pool), table, lens, 4, 2)
    for bad in (pool[..., :-1], pool[0], pool.transpose(0, 2)):
        with pytest.raises(ValueError):
            bd.mx4_shape(bad, table)
        with pytest.raises(ValueError):
            bd.mx4_planes(bad)
    with pytest.raises(ValueError):
        bd.mx4_shape(pool[:, :1].expand(-1, 2, -1), table)


def test_planes_are_views_of_the_records():
    pool = torch.arange(3 * 2 * 17 * 128).remainder(251).to(torch.uint8).reshape(3, 2, 17 * 128)
    view = torch.cat([torch.zeros_like(pool), pool], 1)[:, 2:]  # a strided view with an offset
    for p, q in zip(bd.mx4_planes(pool), bd.mx4_planes(view)):
        assert torch.equal(p, q)
    kc, vc, ks, vs = bd.mx4_planes(view)
    assert kc.shape == vc.shape == (3, 2, 16, 64) and ks.shape == vs.shape == (3, 2, 16, 4)
    assert torch.equal(torch.cat([p.flatten(2) for p in (kc, vc, ks, vs)], 2), pool)
    vs[1, 0, 3, 2] = 252
    assert view[1, 0, 2112 + 3 * 4 + 2] == 252
