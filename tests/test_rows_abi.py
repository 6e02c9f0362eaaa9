"""Refusals of the row-dependent products and the expert routing, without a
GPU: every bad argument is rejected on the host before any CUDA call."""
import ctypes

import pytest
import torch

import weight_only_quantized_rq_b200 as rq

P = ctypes.c_void_p
A, B, U = P(0x40000), P(0x80000), P(0x40004)       # aligned and misaligned fake device addresses (never read)
NULL = P(0)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from weight_only_quantized_rq_b200 import build
    build.build()
    return rq.lib()


def _desc(fmt, K, N, scales=0x20000):
    return rq.RqPacked(rq.fmt_id(fmt), K, N, 0, 0x10000, scales)


def _grouped(L, x=A, T=4, K=256, N=32, w=None, E=4, R=8, offsets=0x50000, in_rows=0, out_rows=0, y=B, Ty=8, act=0,
             out=0, ws=B, size=BIG):
    w = _desc("w4g64", 256, 128) if w is None else w
    g = rq.RqGroups(E, R, offsets, in_rows, out_rows)
    return L.rq_wgemm_grouped(x, T, K, N, w, g, y, Ty, act, out, ws, size, NULL)


@pytest.mark.parametrize("change,status", [
    (dict(x=NULL), rq.RQ_ERR_INVALID_ARG),
    (dict(y=NULL), rq.RQ_ERR_INVALID_ARG),
    (dict(ws=NULL), rq.RQ_ERR_INVALID_ARG),
    (dict(offsets=0), rq.RQ_ERR_INVALID_ARG),
    (dict(T=0), rq.RQ_ERR_INVALID_ARG),
    (dict(T=(1 << 20) + 1), rq.RQ_ERR_INVALID_ARG),
    (dict(Ty=0), rq.RQ_ERR_INVALID_ARG),
    (dict(R=0), rq.RQ_ERR_INVALID_ARG),
    (dict(R=(1 << 20) + 1), rq.RQ_ERR_INVALID_ARG),
    (dict(E=0), rq.RQ_ERR_INVALID_ARG),
    (dict(E=1025), rq.RQ_ERR_INVALID_ARG),
    (dict(N=0), rq.RQ_ERR_INVALID_ARG),
    (dict(N=(1 << 24) // 4 + 1), rq.RQ_ERR_INVALID_ARG),
    (dict(N=31), rq.RQ_ERR_FORMAT_MISMATCH),
    (dict(E=2), rq.RQ_ERR_FORMAT_MISMATCH),
    (dict(K=192), rq.RQ_ERR_FORMAT_MISMATCH),
    (dict(w=_desc("w4g64", 96, 128)), rq.RQ_ERR_UNSUPPORTED_SHAPE),
    (dict(w=_desc("w4sb32", 256, 128)), rq.RQ_ERR_FORMAT_MISMATCH),
    (dict(act=2), rq.RQ_ERR_INVALID_ARG),
    (dict(out=2), rq.RQ_ERR_INVALID_ARG),
    (dict(x=U), rq.RQ_ERR_MISALIGNED),
    (dict(y=U), rq.RQ_ERR_MISALIGNED),
    (dict(ws=U), rq.RQ_ERR_MISALIGNED),
    (dict(offsets=0x50004), rq.RQ_ERR_MISALIGNED),
    (dict(in_rows=0x50004), rq.RQ_ERR_MISALIGNED),
    (dict(out_rows=0x50004), rq.RQ_ERR_MISALIGNED),
    (dict(size=15), rq.RQ_ERR_INVALID_ARG),
])
def test_grouped_refuses(L, change, status):
    assert _grouped(L, **change) == status


def test_grouped_workspace_size(L):
    for fmt in rq.FORMAT_IDS:
        assert L.rq_grouped_workspace_size(rq.fmt_id(fmt), 8, 512, 40, 4) > 0
    f = rq.fmt_id("w4g64")
    for bad in ((0, 8, 512, 40, 4), (f, 0, 512, 40, 4), (f, 8, 96, 40, 4), (f, 8, 512, 0, 4), (f, 8, 512, 40, 0),
                (f, 8, 512, 1 << 23, 4), (f, (1 << 20) + 1, 512, 40, 4), (f, 8, 512, 40, 1025)):
        assert L.rq_grouped_workspace_size(*bad) == 0


def _lora(L, x=A, M=4, K=256, N=32, w=None, n=2, rank=16, a=0x50000, b=0x60000, scales=0x70000, ranks=0, rows=A, y=B,
          out=0, ws=B, size=BIG):
    w = _desc("w4g64", 256, 32) if w is None else w
    ad = rq.RqLora(n, rank, a, b, scales, ranks)
    return L.rq_wgemm_lora(x, M, K, N, w, ad, rows, y, out, ws, size, NULL)


@pytest.mark.parametrize("change,status", [
    (dict(x=NULL), rq.RQ_ERR_INVALID_ARG),
    (dict(rows=NULL), rq.RQ_ERR_INVALID_ARG),
    (dict(y=NULL), rq.RQ_ERR_INVALID_ARG),
    (dict(ws=NULL), rq.RQ_ERR_INVALID_ARG),
    (dict(a=0), rq.RQ_ERR_INVALID_ARG),
    (dict(b=0), rq.RQ_ERR_INVALID_ARG),
    (dict(scales=0), rq.RQ_ERR_INVALID_ARG),
    (dict(M=0), rq.RQ_ERR_INVALID_ARG),
    (dict(n=0), rq.RQ_ERR_INVALID_ARG),
    (dict(out=5), rq.RQ_ERR_INVALID_ARG),
    (dict(rank=12), rq.RQ_ERR_UNSUPPORTED_SHAPE),
    (dict(rank=0), rq.RQ_ERR_UNSUPPORTED_SHAPE),
    (dict(rank=264), rq.RQ_ERR_UNSUPPORTED_SHAPE),
    (dict(K=512), rq.RQ_ERR_FORMAT_MISMATCH),
    (dict(x=U), rq.RQ_ERR_MISALIGNED),
    (dict(a=0x50008), rq.RQ_ERR_MISALIGNED),
    (dict(ranks=0x50008), rq.RQ_ERR_MISALIGNED),
    (dict(rows=U), rq.RQ_ERR_MISALIGNED),
    (dict(size=0), rq.RQ_ERR_INVALID_ARG),
])
def test_lora_refuses(L, change, status):
    assert _lora(L, **change) == status


def _route(L, logits=A, kind=0, T=4, E=8, k=2, renorm=0, ids=0x50000, w=0x51000, off=0x52000, rows=0x53000,
           slots=0x54000, ws=B, size=BIG):
    return L.rq_route_topk(logits, kind, T, E, k, renorm, rq.RqRouting(ids, w, off, rows, slots), ws, size, NULL)


@pytest.mark.parametrize("change,status", [
    (dict(logits=NULL), rq.RQ_ERR_INVALID_ARG),
    (dict(ids=0), rq.RQ_ERR_INVALID_ARG),
    (dict(slots=0), rq.RQ_ERR_INVALID_ARG),
    (dict(kind=2), rq.RQ_ERR_INVALID_ARG),
    (dict(renorm=2), rq.RQ_ERR_INVALID_ARG),
    (dict(T=0), rq.RQ_ERR_INVALID_ARG),
    (dict(E=0), rq.RQ_ERR_INVALID_ARG),
    (dict(E=1025), rq.RQ_ERR_INVALID_ARG),
    (dict(k=0), rq.RQ_ERR_INVALID_ARG),
    (dict(k=9), rq.RQ_ERR_INVALID_ARG),
    (dict(E=64, k=17), rq.RQ_ERR_INVALID_ARG),
    (dict(T=1 << 20, k=2), rq.RQ_ERR_INVALID_ARG),
    (dict(size=0), rq.RQ_ERR_INVALID_ARG),
    (dict(logits=U), rq.RQ_ERR_MISALIGNED),
    (dict(off=0x52004), rq.RQ_ERR_MISALIGNED),
])
def test_route_refuses(L, change, status):
    assert _route(L, **change) == status


@pytest.mark.parametrize("args,status", [
    ((NULL, 0, A, A, 4, 64, 2, B, 0), rq.RQ_ERR_INVALID_ARG),
    ((A, 3, A, A, 4, 64, 2, B, 0), rq.RQ_ERR_INVALID_ARG),
    ((A, 0, A, A, 4, 64, 2, B, 3), rq.RQ_ERR_INVALID_ARG),
    ((A, 0, A, A, 0, 64, 2, B, 0), rq.RQ_ERR_INVALID_ARG),
    ((A, 0, A, A, 4, 0, 2, B, 0), rq.RQ_ERR_INVALID_ARG),
    ((A, 0, A, A, 4, 64, 17, B, 0), rq.RQ_ERR_INVALID_ARG),
    ((A, 0, A, A, 4, 64, 2, U, 0), rq.RQ_ERR_MISALIGNED),
])
def test_combine_refuses(L, args, status):
    assert L.rq_route_combine(*args, NULL) == status


def test_binding_refuses():
    """The Python checks: shapes, dtypes, layout and devices, before the C call."""
    codes, scales = torch.zeros(12 * 128, dtype=torch.uint8), torch.zeros(12 * 8, dtype=torch.uint8)
    w = rq.Packed(rq.fmt_id("w4g64"), 256, 12, codes, scales)
    with pytest.raises(ValueError, match="equal experts"):
        rq.GroupedExperts(w, 5)
    with pytest.raises(rq.RqError):
        rq.GroupedExperts(w, 4, max_rows=0)
    ex = rq.GroupedExperts(w, 4, max_rows=6)
    x, off = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32)
    for bad in (dict(x=x.float()), dict(x=x[:, :128]), dict(x=x.t().contiguous().t()), dict(offsets=off[:4]),
                dict(offsets=off.long()), dict(in_rows=torch.zeros(7, dtype=torch.int32)), dict(act="gelu"),
                dict(in_rows=torch.zeros(2, dtype=torch.int32), out_rows=torch.zeros(3, dtype=torch.int32)),
                dict()):                                        # not on a GPU
        with pytest.raises(ValueError):
            ex(**{**dict(x=x, offsets=off), **bad})
    a, b, s = torch.zeros(2, 16, 256, dtype=torch.bfloat16), torch.zeros(2, 12, 16, dtype=torch.bfloat16), torch.zeros(2)
    for bad in ((a.float(), b, s), (a, b[:, :11], s), (a, b, s[:1]), (a[0], b, s)):
        with pytest.raises(ValueError):
            rq.LoraProjection(w, *bad)
    with pytest.raises(rq.RqError):                             # rank 12
        rq.LoraProjection(w, a[:, :12].contiguous(), b[..., :12].contiguous(), s)
    lp = rq.LoraProjection(w, a, b, s, max_rows=4)
    rows = torch.zeros(4, dtype=torch.int32)
    for bad in (dict(row_adapter=rows.long()), dict(row_adapter=rows[:3]), dict(x=torch.zeros(5, 256, dtype=torch.bfloat16),
                row_adapter=torch.zeros(5, dtype=torch.int32)), dict()):
        with pytest.raises(ValueError):
            lp(**{**dict(x=x, row_adapter=rows), **bad})
    for E, k in ((0, 1), (4, 5), (2000, 2), (64, 17)):
        with pytest.raises(ValueError):
            rq.TopkRouter(E, k)
    for bad in (torch.zeros(3, 8, dtype=torch.float16), torch.zeros(3, 9), torch.zeros(3, 8)):
        with pytest.raises(ValueError):
            rq.TopkRouter(8, 2)(bad)
    with pytest.raises(ValueError):
        rq.rq_route_combine(torch.zeros(6, 4), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2))
