"""Expert routing and the combine on the GPU against plain 64-bit definitions."""
import numpy as np
import pytest
import torch

import weight_only_quantized_rq_b200 as rq

pytestmark = pytest.mark.gpu
DEV = "cuda"


def route_ref(logits, k, renorm):
    l = logits.double().cpu().numpy().copy()
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, float(np.finfo(np.float32).max))
    T, E = l.shape
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        order = np.argsort(-l[t], kind="stable")[:k]
        order = [e for e in order if l[t, e] > -np.inf]
        if not order:
            continue
        p = np.exp(l[t] - l[t].max())
        den = p[order].sum() if renorm else p.sum()
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[order] / den
    flat = ids.reshape(-1)
    slots = np.concatenate([np.nonzero(flat == e)[0] for e in range(E)]).astype(np.int32)
    off = np.concatenate(([0], np.cumsum([(flat == e).sum() for e in range(E)]))).astype(np.int32)
    pad = np.full(T * k - slots.size, -1, np.int32)
    return ids, w, off, np.concatenate((slots // k, pad)), np.concatenate((slots, pad))


def check_route(logits, k, renorm):
    r = rq.rq_route_topk(logits, k, renorm)
    ids, w, off, rows, slots = route_ref(logits, k, renorm)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.in_rows.cpu().numpy(), rows)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    # exp in fp32: 2 ulp of its own, the argument's subtraction 2^-24 |l - max| relative to the result, E additions
    E = logits.shape[1]
    l = logits.double().nan_to_num(neginf=0.0, posinf=0.0).abs().max().item() if logits.numel() else 0.0
    tol = (E + 16 + 4 * min(l, 200.0)) * 2.0 ** -24
    err = np.abs(r.weights.cpu().numpy() - w)
    assert (err <= tol * np.maximum(w, 2.0 ** -100) + 2.0 ** -120).all(), float(err.max())
    return r


@pytest.mark.parametrize("T", [1, 2, 7, 31, 32, 33, 255, 256, 257, 700, 3001])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (8, 2), (64, 4), (65, 1), (256, 8), (1000, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route(T, E, k, dtype):
    g = torch.Generator().manual_seed(T * 31 + E)
    logits = (torch.randn(T, E, generator=g) * 3).to(dtype).to(DEV)      # bf16: many ties
    check_route(logits, k, T % 2 == 0)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_masks(renorm):
    """-inf, NaN, +inf, the type's lowest value, rows that nothing is left of, all equal rows."""
    g = torch.Generator().manual_seed(3)
    l = torch.randn(40, 12, generator=g)
    l[0] = -float("inf")
    l[1] = float("nan")
    l[2, 3:] = -float("inf")
    l[3] = torch.finfo(torch.float32).min
    l[4, 5] = float("inf")
    l[5, 1:4] = float("inf")
    l[6] = 0.0
    l[7, ::2] = float("nan")
    l[8] = torch.finfo(torch.float32).min
    l[8, 7] = -1e38
    l[9, :] = -float("inf")
    l[9, 11] = torch.finfo(torch.float32).min
    l[10, 0], l[10, 1] = 0.0, -0.0
    check_route(l.to(DEV), 4, renorm)


def test_route_all_to_one_expert_and_nothing():
    l = torch.full((513, 16), -float("inf"))
    r = check_route(l.to(DEV), 3, True)
    assert (r.offsets == 0).all()
    l[:, 9] = 1.0
    check_route(l.to(DEV), 3, False)


def test_route_zero_tokens():
    r = rq.rq_route_topk(torch.zeros(0, 8, device=DEV), 2)
    assert r.ids.shape == (0, 2) and (r.offsets == 0).all() and r.offsets.shape == (9,)


def test_route_large():
    g = torch.Generator().manual_seed(9)
    logits = torch.randn(40000, 128, generator=g).to(DEV)
    a = check_route(logits, 8, True)
    b = rq.rq_route_topk(logits, 8, True)
    assert torch.equal(a.weights, b.weights)


def test_route_in_a_graph():
    logits = torch.randn(300, 16, device=DEV)
    router = rq.TopkRouter(16, 2)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        router(logits)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            r = router(logits)
    for seed in range(3):
        logits.copy_(torch.randn(300, 16, generator=torch.Generator().manual_seed(seed)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = route_ref(logits, 2, False)
        assert np.array_equal(r.ids.cpu().numpy(), want[0]) and np.array_equal(r.slots.cpu().numpy(), want[4])


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 2, 7), (32, 2, 2048), (5, 16, 33), (257, 3, 768), (1, 4, 4095)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_combine(T, k, N, dtype, out):
    g = torch.Generator().manual_seed(T + N)
    y = torch.randn(T * k, N, generator=g).to(dtype).to(DEV)
    ids = torch.randint(0, 9, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand(T, k, generator=g) < 0.2] = -1
    ids[T // 2] = -1
    y[ids.view(-1).to(DEV) < 0] = float("nan")          # rows without an expert are never read
    w = torch.randn(T, k, generator=g).to(DEV)
    guard = torch.full((T + 1, N), 7.5, dtype=out, device=DEV)
    rq.rq_route_combine(y, ids.to(DEV), w, out=guard[:T])
    keep = (ids >= 0).to(DEV)
    yd = torch.where(keep.view(-1, 1), y.double(), 0.0).view(T, k, N)
    ref, S = (yd * w.double()[..., None]).sum(1), (yd.abs() * w.double().abs()[..., None]).sum(1)
    tol = k * 2.0 ** -24 * S
    if out == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert ((guard[:T].double() - ref).abs() <= tol).all()
    assert (guard[T] == 7.5).all()


@pytest.mark.parametrize("N", [2056, 4096, 4104, 8200])
@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_combine_wide_rows(N, k, dtype, out):
    """Rows of several blocks, the last one partly filled; what a slot without an expert holds is not used."""
    T = 5
    g = torch.Generator().manual_seed(N + k)
    y = torch.randn(T * k, N, generator=g).to(dtype).to(DEV)
    ids = torch.randint(0, 9, (T, k), generator=g, dtype=torch.int32)
    ids[1, 0] = -1
    ids[3] = -1
    y[ids.view(-1).to(DEV) < 0] = float("nan")
    w = torch.randn(T, k, generator=g).to(DEV)
    guard = torch.full((T + 1, N), 7.5, dtype=out, device=DEV)
    rq.rq_route_combine(y, ids.to(DEV), w, out=guard[:T])
    yd = torch.where((ids >= 0).to(DEV).view(-1, 1), y.double(), 0.0).view(T, k, N)
    ref, S = (yd * w.double()[..., None]).sum(1), (yd.abs() * w.double().abs()[..., None]).sum(1)
    tol = k * 2.0 ** -24 * S                             # k products, each added with one rounding
    if out == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert ((guard[:T].double() - ref).abs() <= tol).all()
    assert (guard[T] == 7.5).all()
