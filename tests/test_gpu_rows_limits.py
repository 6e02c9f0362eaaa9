"""Row-dependent products and routing at their limits: waits that run out,
the largest tables, captured adapter calls, shared objects on several streams."""
import numpy as np
import pytest
import torch

import weight_only_quantized_rq_b200 as rq
from test_gpu_rows import DEV, check, grouped_ref, random_packed, rows_of

pytestmark = pytest.mark.gpu
WAIT_BITS = 0x1F          # copy, slot, commit and TMEM waits


def adapters(n, r, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    A = (torch.randn(n, r, K, generator=g) / K ** 0.5).to(torch.bfloat16).to(DEV)
    B = torch.randn(n, N, r, generator=g).to(torch.bfloat16).to(DEV)
    return A, B, torch.linspace(0.5, 2.0, n, device=DEV)


@pytest.mark.parametrize("M,dtype,kind", [
    (8, torch.float32, "grouped"), (40, torch.float32, "grouped"), (400, torch.bfloat16, "grouped"),
    (4, torch.float32, "lora"), (20, torch.float32, "lora"), (130, torch.bfloat16, "lora")])
def test_waits_run_out_then_the_next_call_is_correct(orc, M, dtype, kind):
    """Copies that are never issued: every wait gives up after 1 ms, the status word says so, the next call is right."""
    K, N = 1024, 700
    x = rows_of(M, K, 50)
    if kind == "grouped":
        w, _ = random_packed(orc, "w4g64", 2 * N, K, 50)
        ex, off = rq.GroupedExperts(w, 2, M), torch.tensor([0, M // 2, M], dtype=torch.int32, device=DEV)
        call = lambda: ex(x, off, out_dtype=dtype)
    else:
        w, _ = random_packed(orc, "w4g64", N, K, 50)
        lp, row = rq.LoraProjection(w, *adapters(3, 16, K, N, 50), max_rows=M), torch.arange(M, dtype=torch.int32, device=DEV) % 4 - 1
        call = lambda: lp(x, row, out_dtype=dtype)
    want = call()
    assert rq.rq_device_status() == 0
    try:
        rq.rq_test_hooks(1_000_000, 1)
        call()
        word = rq.rq_device_status()
    finally:
        rq.rq_test_hooks(0, 0)
    assert word & WAIT_BITS, word
    assert rq.rq_device_status() == 0
    assert torch.equal(call(), want)
    assert rq.rq_device_status() == 0


@pytest.mark.parametrize("fmt", ["w4g64", "w8g16", "w6sb32"])
@pytest.mark.parametrize("rows,dtype", [(700, torch.bfloat16), (17000, torch.bfloat16), (700, torch.float32)])
def test_most_experts(orc, fmt, rows, dtype):
    """1024 experts, most of them with no or few rows, some with many."""
    E, N, K = 1024, 24, 256
    w, What = random_packed(orc, fmt, E * N, K, 51)
    r = np.random.default_rng(rows)
    off = np.sort(np.concatenate(([0], r.integers(0, rows + 1, E - 1), [rows]))).astype(np.int32)
    off[300:500] = off[300]                              # a long run of empty groups, then a large one
    x = rows_of(rows, K, 51)
    y = rq.rq_wgemm_grouped(x, w, torch.from_numpy(off).to(DEV), out_dtype=dtype)
    ref = grouped_ref(x, What, E, off, None)
    live = sorted(ref)
    check(y[live], torch.stack([ref[i][0] for i in live]), torch.stack([ref[i][1] for i in live]), K)


@pytest.mark.parametrize("T,E,k", [(131072, 8, 8), (65536, 1024, 16), (1 << 20, 3, 1)])
def test_route_most_pairs(T, E, k):
    """2^20 pairs: the grouping is the stable sort of the pairs by expert, the choices are the largest logits."""
    logits = torch.randn(T, E, device=DEV, generator=torch.Generator(DEV).manual_seed(5))
    r = rq.rq_route_topk(logits, k, True)
    ids = r.ids.view(-1).long()
    order = torch.sort(ids, stable=True).indices
    assert torch.equal(r.slots.long(), order) and torch.equal(r.in_rows.long(), order // k)
    assert torch.equal(r.offsets.long(), torch.searchsorted(ids[order], torch.arange(E + 1, device=DEV)))
    got = torch.gather(logits, 1, r.ids.long())
    assert torch.equal(got, torch.topk(logits, k).values)


@pytest.mark.parametrize("M,dtype", [(3, torch.float32), (24, torch.float32), (70, torch.bfloat16), (1100, torch.bfloat16)])
def test_lora_graph_replays_with_new_adapters(orc, M, dtype):
    """A captured call replays with the rows and adapters of the moment, beside eager calls of the same object."""
    K, N, n = 512, 200, 5
    w, _ = random_packed(orc, "w8g64", N, K, 52)
    lp = rq.LoraProjection(w, *adapters(n, 24, K, N, 52), max_rows=M)
    x, row = rows_of(M, K, 52), torch.full((M,), -1, dtype=torch.int32, device=DEV)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        lp(x, row, out_dtype=dtype)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            y = lp(x, row, out_dtype=dtype)
    for seed in range(3):
        gen = torch.Generator().manual_seed(seed)
        row.copy_(torch.randint(-1, n + 1, (M,), generator=gen, dtype=torch.int32))
        x.copy_(rows_of(M, K, 60 + seed))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        eager = lp(x, row, out_dtype=dtype)              # on another stream, at the same time
        torch.cuda.synchronize()
        assert torch.equal(eager, y)


@pytest.mark.parametrize("M,dtype", [(5, torch.float32), (30, torch.float32), (130, torch.bfloat16)])
def test_lora_two_streams_and_two_graphs_at_once(orc, M, dtype):
    K, N = 1024, 320
    w, _ = random_packed(orc, "w4sb32", N, K, 53)
    lp = rq.LoraProjection(w, *adapters(4, 16, K, N, 53), max_rows=M)
    xs = [rows_of(M, K, 70 + i) for i in range(2)]
    rows = [torch.arange(M, dtype=torch.int32, device=DEV) % (3 + i) for i in range(2)]
    want = [lp(x, r, out_dtype=dtype) for x, r in zip(xs, rows)]
    streams, graphs, got = [torch.cuda.Stream() for _ in range(2)], [], []
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            got.append(lp(xs[i], rows[i], out_dtype=dtype))
        graphs.append(g)
    eager = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
                eager[i].append(lp(xs[i], rows[i], out_dtype=dtype))
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i], want[i]) and all(torch.equal(e, want[i]) for e in eager[i])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_same_row_read_by_many_and_rows_behind_stay(orc, dtype):
    """in_rows may name a row any number of times; rows of y that no index names stay as they were."""
    K, N, E = 256, 136, 2
    w, What = random_packed(orc, "w4g64", E * N, K, 54)
    x = rows_of(3, K, 54)
    src = np.array([1, 1, 1, 2] * 20, np.int32)
    off = np.array([0, 50, 80], np.int32)
    dst = np.arange(80, dtype=np.int32)[::-1].copy() + 5
    y = torch.full((90, N), 7.5, dtype=dtype, device=DEV)
    rq.rq_wgemm_grouped(x, w, torch.from_numpy(off).to(DEV), in_rows=torch.from_numpy(src).to(DEV),
                        out_rows=torch.from_numpy(dst).to(DEV), y=y)
    ref = grouped_ref(x, What, E, off, src)
    check(y[torch.from_numpy(dst).long().to(DEV)], torch.stack([ref[i][0] for i in range(80)]), torch.stack([ref[i][1] for i in range(80)]), K)
    assert (y[:5] == 7.5).all() and (y[85:] == 7.5).all()


@pytest.mark.parametrize("M,dtype", [(5, torch.float32), (20, torch.float32), (70, torch.bfloat16)])
def test_lora_nonfinite_adapter_stays_with_its_rows(orc, M, dtype):
    """Infinities and NaN in one adapter reach only the rows that use it, whatever shares a tile with them."""
    K, N = 512, 136
    w, _ = random_packed(orc, "w4g64", N, K, 55)
    A, B, sc = adapters(4, 40, K, N, 55)
    x, row = rows_of(M, K, 55), torch.arange(M, dtype=torch.int32, device=DEV) % 5 - 1
    want = rq.rq_wgemm_lora(x, w, A, B, sc, row, out_dtype=dtype)
    A[1, 3, 5], A[2, 39, 0], B[1, 7], B[2, :, 39], B[2, 100, 0] = float("nan"), float("inf"), float("inf"), -float("inf"), float("nan")
    got = rq.rq_wgemm_lora(x, w, A, B, sc, row, out_dtype=dtype)
    hit = (row == 1) | (row == 2)
    assert torch.equal(got[~hit], want[~hit])
    assert not torch.isfinite(got[row == 1][:, 7]).any() and not torch.isfinite(got[row == 2]).any()


@pytest.mark.parametrize("fmt", ["w4sb32", "w6sb32"])
def test_superblocks_that_cancel(orc, fmt):
    """Weights S u - M far below M: many-row bf16 results are within 2^-11 of the sums of |x| (S u + |M|), as
    S and M are rounded to fp16 (2^-12 each), fp32 results within fp32's bound of them."""
    K, N, M, size = 512, 200, 96, {"w4sb32": 144, "w6sb32": 208}[fmt]
    r = np.random.default_rng(56)
    rec = r.integers(0, 256, (N, K // 256, size), dtype=np.uint8)
    rec[..., 4:16] = 0xFF                               # group scales and minima at their largest
    d = (r.uniform(0.5, 1.5, (N, K // 256)) * 1e-4).astype(np.float16)
    def packed(dmin):
        rec[..., :4] = np.stack([d, dmin.astype(np.float16)], -1).view(np.uint8)
        codes = rec.reshape(-1).copy()
        return codes, torch.from_numpy(np.asarray(orc.dequant(fmt, K, N, codes, None)).reshape(N, K)).to(DEV).double()
    _, Su = packed(np.zeros_like(d))
    codes, What = packed(d.astype(np.float32) * (7.5 if fmt == "w4sb32" else 31.5))
    w = rq.Packed(rq.fmt_id(fmt), K, N, torch.from_numpy(codes).to(DEV), None)
    x = rows_of(M, K, 56)
    xd = x.double()
    off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    wide = xd.abs() @ (Su + (Su - What).abs()).t()
    for dtype in (torch.float32, torch.bfloat16):
        y = rq.rq_wgemm_grouped(x, w, off, out_dtype=dtype)
        check(y, xd @ What.t(), wide, K)


def test_many_rows_with_indices_out_of_range_and_not_finite(orc):
    """Many-row bf16 products: rows of x that do not exist, rows of y that do not, duplicates, infinities and NaN."""
    E, N, K, R = 3, 264, 320, 150
    w, What = random_packed(orc, "w8g64", E * N, K, 57)
    x = rows_of(40, K, 57)
    x[3, 7], x[9, 300] = float("inf"), float("nan")
    r = np.random.default_rng(57)
    src = r.integers(-2, 43, R).astype(np.int32)
    dst = r.permutation(R + 10)[:R].astype(np.int32)
    dst[::17] = -1
    dst[5::31] = 1 << 30
    raw = np.array([3, 70, 60, 400], np.int32)
    off = np.minimum(np.maximum.accumulate(raw), R)
    y = torch.full((R + 10, N), 7.5, dtype=torch.bfloat16, device=DEV)
    t = lambda a: torch.from_numpy(a).to(DEV)
    rq.rq_wgemm_grouped(x, w, t(raw), t(src), t(dst), y=y)
    ref = grouped_ref(torch.where(torch.isfinite(x), x, 0), What, E, off, src)
    stored = [i for i in sorted(ref) if 0 <= dst[i] < R + 10]
    good, bad = [i for i in stored if src[i] not in (3, 9)], [i for i in stored if src[i] in (3, 9)]
    check(y[[int(dst[i]) for i in good]], torch.stack([ref[i][0] for i in good]), torch.stack([ref[i][1] for i in good]), K)
    assert bad and not torch.isfinite(y[[int(dst[i]) for i in bad]]).any()
    rest = sorted(set(range(R + 10)) - {int(dst[i]) for i in stored})
    assert (y[rest] == 7.5).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_offsets_past_32_bits(orc, dtype):
    """The most rows, x and y of more than 2^31 elements, indices at their ends; then the combine of the rows."""
    E, K, N, R = 2, 2560, 2304, 1 << 20
    w, What = random_packed(orc, "w4g64", E * N, K, 58)
    g = torch.Generator(DEV).manual_seed(58)
    x = torch.empty(R, K, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    off = torch.tensor([0, R - 300001, R], dtype=torch.int32, device=DEV)
    rows = torch.arange(R, dtype=torch.int32, device=DEV)
    y = torch.empty(R, N, dtype=dtype, device=DEV)
    rq.rq_wgemm_grouped(x, w, off, in_rows=R - 1 - rows, out_rows=rows, y=y)
    at = torch.cat([torch.arange(40, device=DEV), torch.randint(0, R, (200,), device=DEV, generator=g), torch.arange(R - 40, R, device=DEV)])
    e = (at >= R - 300001).long()
    v = x[R - 1 - at].double()
    ref, S = torch.empty(len(at), N, dtype=torch.float64, device=DEV), torch.empty(len(at), N, dtype=torch.float64, device=DEV)
    for i in range(E):
        We = What[i * N:(i + 1) * N]
        ref[e == i], S[e == i] = v[e == i] @ We.t(), v[e == i].abs() @ We.abs().t()
    check(y[at], ref, S, K)
    out = rq.rq_route_combine(y, torch.zeros(R // 2, 2, dtype=torch.int32, device=DEV), torch.ones(R // 2, 2, device=DEV), out_dtype=torch.float32)
    t = at // 2
    want = y[2 * t].double() + y[2 * t + 1].double()
    assert ((out[t].double() - want).abs() <= 2.0 ** -23 * (y[2 * t].double().abs() + y[2 * t + 1].double().abs())).all()
    one = rq.Packed(w.fmt, K, N, w.codes[:w.codes.numel() // E].clone(), w.scales[:N * (K // 64) * 2].clone())
    A, B, sc = adapters(3, 8, K, N, 58)
    rq.LoraProjection(one, A, B, sc, max_rows=R)(x, rows % 4 - 1, y=y)
    v, a = x[at].double(), at % 4 - 1
    ref, S, extra = v @ What[:N].t(), v.abs() @ What[:N].abs().t(), torch.zeros_like(ref)
    for i in range(3):
        Ad, Bd, m = A[i].double(), B[i].double(), a == i
        ref[m] += float(sc[i]) * (v[m] @ Ad.t()) @ Bd.t()
        extra[m] = (K + 12) * 2.0 ** -23 * float(sc[i]) * (v[m].abs() @ Ad.abs().t()) @ Bd.abs().t()
    check(y[at], ref, S, K, extra=extra)
    assert rq.rq_device_status() == 0
