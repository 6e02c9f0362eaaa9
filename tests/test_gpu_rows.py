"""Products grouped by expert and adapters beside a packed projection, on the
GPU, against sums in 64 bits over the oracle's dequantized weights.

Bounds (derived, not fitted): a sum of n products in fp32 in any order is
within n 2^-24 S of the exact one, S = sum |x| |w_hat| (twice that where the
adder truncates instead of rounding); w_hat itself is one fp32 rounding off
for the superblocks, and the bf16 results may be computed with weights and
activations rounded to 11 bits (2^-11 S, twice). A bf16 result adds half a
step of its own. The adapter's term adds its two sums: (K + r) 2^-23 of the
absolute sums.
"""
import numpy as np
import pytest
import torch

import weight_only_quantized_rq_b200 as rq

pytestmark = pytest.mark.gpu
DEV = "cuda"
SB = {"w4sb32": 144, "w5sb32": 176, "w6sb32": 208}
FORMATS = tuple(rq.FORMAT_IDS)


def random_packed(orc, fmt, rows, K, seed):
    """A Packed of random valid codes and its w_hat in 64 bits (on the GPU)."""
    r = np.random.default_rng(seed)
    if fmt in SB:
        rec = r.integers(0, 256, (rows, K // 256, SB[fmt]), dtype=np.uint8)
        head = (r.uniform(0.5, 1.5, (rows, K // 256, 2)) * [3e-4, 2e-3]).astype(np.float16)
        rec[..., :4] = head.view(np.uint8)
        codes, scales = rec.reshape(-1), None
    else:
        cb, sb = rq.rq_packed_size(fmt, K, rows)
        G = 64 if fmt.endswith("g64") else 16
        if fmt == "w4g64":
            q = r.integers(1, 16, (rows, K), dtype=np.uint8)
            codes = (q[:, 0::2] | (q[:, 1::2] << 4)).reshape(-1)
        elif fmt == "w6g16":
            codes = r.integers(0, 256, cb, dtype=np.uint8)
        else:
            codes = r.integers(1, 256, cb, dtype=np.uint8)
        s = (r.uniform(0.5, 1.5, rows * (K // G)) * 3e-3).astype(np.float16)
        scales = np.zeros(sb, np.uint8)
        scales[:s.size * 2] = s.view(np.uint8)
    w = rq.Packed(rq.fmt_id(fmt), K, rows, torch.from_numpy(codes).to(DEV),
                  None if scales is None else torch.from_numpy(scales).to(DEV))
    osc = None if scales is None else scales[:s.size * 2].view(np.uint16)
    w_hat = orc.dequant(fmt, K, rows, codes, osc)
    return w, torch.from_numpy(np.asarray(w_hat).reshape(rows, K)).to(DEV).double()


def rows_of(T, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g)
    x[:, 3::97] *= 20
    return x.to(torch.bfloat16).to(DEV)


def check(y, ref, S, K, extra=None, act=None):
    """|y - ref| within the bound of the module's docstring; ref and S before the activation."""
    tol = K * 2.0 ** -23 * S + 2.0 ** -24 * S
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -10 * S
    if extra is not None:
        tol = tol + extra
    if act == "relu2":
        tol = 2 * ref.abs() * tol + tol * tol + 2.0 ** -23 * ref * ref
        ref = ref.clamp(min=0) ** 2
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (y.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol.clamp(min=1e-300)).max()))


def grouped_ref(x, What, E, offsets, in_rows):
    """Exact rows and absolute sums of every row of every group: {row: (y, S)}."""
    N = What.shape[0] // E
    out = {}
    x = x.double()
    for e in range(E):
        idx = list(range(offsets[e], offsets[e + 1]))
        if not idx:
            continue
        src = torch.tensor([in_rows[i] if in_rows is not None else i for i in idx], device=DEV)
        ok = (src >= 0) & (src < x.shape[0])
        xe = torch.where(ok[:, None], x[src.clamp(0, x.shape[0] - 1)], 0.0)
        We = What[e * N:(e + 1) * N]
        y, S = xe @ We.t(), xe.abs() @ We.abs().t()
        for j, i in enumerate(idx):
            out[i] = (y[j], S[j])
    return out


def run_grouped(orc, fmt, K, N, sizes, T=None, gather=False, scatter=False, act=None, dtype=torch.float32, seed=1,
                tail=0):
    E = len(sizes)
    w, What = random_packed(orc, fmt, E * N, K, seed)
    off = np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)
    live = int(off[-1])
    R = live + tail
    rng = np.random.default_rng(seed + 5)
    T = T or max(R, 1)
    x = rows_of(T, K, seed)
    in_rows = rng.integers(0, T, R).astype(np.int32) if gather else None
    out_rows = rng.permutation(R + 3)[:R].astype(np.int32) if scatter else None
    Ty = R + 3 if scatter else max(R, 1)
    y = torch.full((Ty + 2, N), 7.5, dtype=dtype, device=DEV)
    t = lambda a: None if a is None else torch.from_numpy(a).to(DEV)
    rq.GroupedExperts(w, E, max_rows=max(R, 1))(x, t(off), in_rows=t(in_rows), out_rows=t(out_rows), y=y[:Ty], act=act)
    assert rq.rq_device_status() == 0
    ref = grouped_ref(x, What, E, off, in_rows)
    at = {i: int(out_rows[i]) if scatter else i for i in ref}
    if ref:
        rows = sorted(ref)
        check(y[[at[i] for i in rows]], torch.stack([ref[i][0] for i in rows]), torch.stack([ref[i][1] for i in rows]), K,
              act=act)
    untouched = sorted(set(range(Ty + 2)) - set(at.values()))
    assert (y[untouched] == 7.5).all()                 # rows no group names, and the guard rows, keep their values
    return y


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped_formats(orc, fmt, dtype):
    run_grouped(orc, fmt, 512, 200, [3, 0, 1, 9, 17, 0], gather=True, scatter=True, dtype=dtype)


@pytest.mark.parametrize("fmt,K", [("w4g64", 64), ("w4g64", 320), ("w4g64", 768), ("w8g16", 64), ("w8g16", 192),
                                   ("w8g64", 64), ("w8g64", 448), ("w6g16", 64), ("w6g16", 832), ("w4sb32", 256),
                                   ("w4sb32", 2560), ("w5sb32", 768), ("w6sb32", 256), ("w4g64", 8192), ("w8g16", 4096)])
@pytest.mark.parametrize("sizes", [[1], [2, 5]])
def test_grouped_widths(orc, fmt, K, sizes):
    run_grouped(orc, fmt, K, 72, sizes, seed=3)


@pytest.mark.parametrize("N", [1, 7, 16, 127, 128, 129, 300])
@pytest.mark.parametrize("fmt", ["w4g64", "w8g16", "w4sb32"])
def test_grouped_output_widths(orc, fmt, N):
    run_grouped(orc, fmt, 256, N, [4, 1, 11], gather=True, seed=4)


@pytest.mark.parametrize("sizes", [[0, 0, 0], [0], [0, 1], [8, 8, 8], [9, 7, 16, 33], [31, 32, 33], [64, 0, 65], [130, 1],
                                   [1] * 40, [0] * 200 + [3] + [0] * 100])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped_ragged(orc, sizes, dtype):
    run_grouped(orc, "w4g64", 256, 144, sizes, gather=True, tail=5, dtype=dtype, seed=6)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes", [[700, 0, 263], [256, 128, 512, 1]])
def test_grouped_long(orc, fmt, sizes):
    """Prompt-sized groups, bf16 results."""
    run_grouped(orc, fmt, 512, 264, sizes, gather=True, scatter=True, dtype=torch.bfloat16, seed=8)
    run_grouped(orc, fmt, 512, 264, sizes, act="relu2", dtype=torch.bfloat16, seed=9)


@pytest.mark.parametrize("fmt,K", [("w4g64", 64), ("w4g64", 320), ("w4g64", 4096), ("w8g16", 64), ("w8g16", 192), ("w8g64", 448),
                                   ("w6g16", 64), ("w6g16", 832), ("w4sb32", 256), ("w5sb32", 768), ("w6sb32", 512)])
@pytest.mark.parametrize("sizes,N", [([40, 33], 72), ([24], 1), ([25, 200, 0], 129), ([300, 129], 130)])
def test_grouped_many_rows(orc, fmt, K, sizes, N):
    """Groups long enough for the tensor-memory kernel: few tiles (units cut among CTAs), odd widths, K with a ragged end."""
    run_grouped(orc, fmt, K, N, sizes, gather=True, tail=3, dtype=torch.bfloat16, seed=14)


def test_grouped_many_rows_extremes(orc):
    """Rows of very different sizes, tiny, huge, zero and not finite, beside one another in a tile."""
    w, What = random_packed(orc, "w8g16", 2 * 136, 256, 15)
    x = rows_of(60, 256, 15)
    x *= (2.0 ** torch.linspace(-100, 100, 60)).to(torch.bfloat16).to(DEV)[:, None]
    x[7] = 0.0
    x[11, 3], x[40, 255] = float("inf"), float("nan")
    off = torch.tensor([0, 27, 60], dtype=torch.int32, device=DEV)
    y = rq.rq_wgemm_grouped(x, w, off, out_dtype=torch.bfloat16)
    good = [i for i in range(60) if i not in (11, 40)]
    ref = grouped_ref(x, What, 2, [0, 27, 60], None)
    check(y[good], torch.stack([ref[i][0] for i in good]), torch.stack([ref[i][1] for i in good]), 256)
    assert not torch.isfinite(y[[11, 40]]).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped_relu2(orc, dtype):
    run_grouped(orc, "w4g64", 512, 96, [5, 20, 0, 2], act="relu2", dtype=dtype, seed=10)


def test_grouped_index_out_of_range(orc):
    """Offsets out of order or range, rows of x and y that do not exist."""
    E, N, K, R = 4, 40, 256, 12
    w, What = random_packed(orc, "w4g64", E * N, K, 11)
    x = rows_of(6, K, 11)
    raw = np.array([2, -5, 7, 5, 90], np.int32)
    clean = np.minimum(np.maximum.accumulate(np.maximum(raw, 0)), R)
    in_rows = np.array([0, 1, 2, 3, -1, 6, 5, 1 << 30, 0, 1, 2, -(1 << 31)], np.int64).astype(np.int32)
    out_rows = np.array([0, 1, 2, 99, 4, 5, -1, 7, 8, 9, 10, 11], np.int32)
    y = torch.full((12, N), 7.5, device=DEV)
    t = lambda a: torch.from_numpy(a).to(DEV)
    rq.rq_wgemm_grouped(x, w, t(raw), t(in_rows), t(out_rows), y=y)
    ref = grouped_ref(x, What, E, clean, in_rows)
    stored = [i for i in ref if 0 <= out_rows[i] < 12]
    check(y[[int(out_rows[i]) for i in stored]], torch.stack([ref[i][0] for i in stored]),
          torch.stack([ref[i][1] for i in stored]), K)
    rest = sorted(set(range(12)) - {int(out_rows[i]) for i in stored})
    assert (y[rest] == 7.5).all()


def test_grouped_nonfinite_rows_stay_apart(orc):
    """inf and NaN in one row of x reach that row's y only, in every place of a tile."""
    w, What = random_packed(orc, "w4g64", 3 * 64, 256, 12)
    x = rows_of(20, 256, 12)
    x[4, 17], x[9, 200], x[13, 0] = float("inf"), float("nan"), -float("inf")
    off = torch.tensor([0, 6, 12, 20], dtype=torch.int32, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        y = rq.rq_wgemm_grouped(x, w, off, out_dtype=dtype)
        good = [i for i in range(20) if i not in (4, 9, 13)]
        ref = grouped_ref(x, What, 3, [0, 6, 12, 20], None)
        check(y[good], torch.stack([ref[i][0] for i in good]), torch.stack([ref[i][1] for i in good]), 256)
        assert not torch.isfinite(y[[4, 9, 13]]).any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_grouped_is_deterministic_and_matches_itself(orc, fmt):
    """The same rows give the same bits from call to call."""
    w, _ = random_packed(orc, fmt, 4 * 520, 1024, 13)
    x = rows_of(50, 1024, 13)
    off = torch.tensor([0, 1, 30, 30, 50], dtype=torch.int32, device=DEV)
    ex = rq.GroupedExperts(w, 4, 50)
    a = ex(x, off)
    for _ in range(5):
        assert torch.equal(a, ex(x, off))


# ------------------------------------------------------------------ adapters
def run_lora(orc, fmt, M, K, N, n, r, rows=None, ranks=None, dtype=torch.float32, seed=21):
    w, What = random_packed(orc, fmt, N, K, seed)
    x = rows_of(M, K, seed)
    g = torch.Generator().manual_seed(seed)
    A = (torch.randn(n, r, K, generator=g) / K ** 0.5).to(torch.bfloat16).to(DEV)
    B = torch.randn(n, N, r, generator=g).to(torch.bfloat16).to(DEV)
    sc = (torch.rand(n, generator=g) + 0.5).to(DEV)
    rk = [r] * n if ranks is None else list(ranks)
    for a in range(n):                                 # what lies past an adapter's rank never counts
        A[a, max(0, rk[a]):] = float("nan")
        B[a, :, max(0, rk[a]):] = float("nan")
    rows = np.random.default_rng(seed).integers(-1, n + 1, M) if rows is None else np.asarray(rows)
    y = torch.full((M + 2, N), 7.5, dtype=dtype, device=DEV)
    rq.LoraProjection(w, A, B, sc, None if ranks is None else torch.tensor(rk, dtype=torch.int32, device=DEV), M)(
        x, torch.from_numpy(rows.astype(np.int32)).to(DEV), y=y[:M])
    assert rq.rq_device_status() == 0
    xd = x.double()
    ref, S = xd @ What.t(), xd.abs() @ What.abs().t()
    extra = torch.zeros_like(ref)
    for m, a in enumerate(rows):
        k = min(r, max(0, rk[a])) if 0 <= a < n else 0
        if k:
            Ad, Bd, s = A[a, :k].double(), B[a, :, :k].double(), float(sc[a])
            ref[m] += s * (Bd @ (Ad @ xd[m]))
            extra[m] = (K + r + 4) * 2.0 ** -23 * s * (Bd.abs() @ (Ad.abs() @ xd[m].abs()))
    check(y[:M], ref, S, K, extra=extra)
    assert (y[M:] == 7.5).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,dtype", [(1, torch.float32), (5, torch.bfloat16), (19, torch.float32)])
def test_lora_formats(orc, fmt, M, dtype):
    run_lora(orc, fmt, M, 512, 200, 5, 16, dtype=dtype)


@pytest.mark.parametrize("M", [1, 2, 8, 9, 16, 17, 33, 64, 100, 128, 300])
@pytest.mark.parametrize("r", [8, 24, 64])
def test_lora_rows_and_ranks(orc, M, r):
    run_lora(orc, "w4g64", M, 256, 136, 7, r, seed=22)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [9, 32, 70, 129])
def test_lora_many_rows(orc, fmt, M):
    """bf16 results above the few rows whose adapters the product itself does, on either product kernel."""
    run_lora(orc, fmt, M, 512, 200, 5, 40, ranks=[40, 0, 13, 33, 8], dtype=torch.bfloat16, seed=27)


def test_lora_rounds_of_rows(orc):
    """More rows than one round of launches takes."""
    for dtype in (torch.float32, torch.bfloat16):
        run_lora(orc, "w4g64", 2050, 128, 72, 9, 16, dtype=dtype, seed=28)


@pytest.mark.parametrize("K,N", [(64, 1), (192, 129), (4096, 96), (8192, 40)])
@pytest.mark.parametrize("fmt", ["w4g64", "w8g16"])
def test_lora_widths(orc, fmt, K, N):
    run_lora(orc, fmt, 6, K, N, 3, 32, seed=23)


def test_lora_ragged_ranks_and_rows(orc):
    """Ranks of 0, odd, full and beyond the slot, rows without an adapter or with no such slot."""
    run_lora(orc, "w4sb32", 12, 512, 260, 6, 40, rows=[0, 1, 2, 3, 4, 5, -1, 6, 1 << 30, 2, 2, -(1 << 31)],
             ranks=[0, 1, 40, 39, 64, -3], dtype=torch.bfloat16, seed=24)


def test_lora_no_row_has_an_adapter(orc):
    run_lora(orc, "w8g64", 4, 256, 64, 2, 16, rows=[-1, -1, 9, -1], seed=25)


def test_lora_largest_rank_one_adapter_for_all(orc):
    run_lora(orc, "w4g64", 40, 512, 200, 1, 256, rows=[0] * 40, seed=26)


# ------------------------------------------------------- streams and graphs
def test_two_streams_at_once(orc):
    """Calls of one prepared object on two streams do not share a workspace."""
    w, _ = random_packed(orc, "w4g64", 4 * 256, 512, 31)
    ex = rq.GroupedExperts(w, 4, 64)
    x = [rows_of(64, 512, 40 + i) for i in range(2)]
    off = torch.tensor([0, 10, 20, 50, 64], dtype=torch.int32, device=DEV)
    want = [ex(v, off) for v in x]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(ex(x[i], off))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], g) for g in got[i])


def test_stream_argument(orc):
    """A stream of the caller's choice, its work ordered with the caller's own on it."""
    w, _ = random_packed(orc, "w4g64", 200, 512, 32)
    A = torch.randn(2, 8, 512, device=DEV).to(torch.bfloat16)
    B = torch.randn(2, 200, 8, device=DEV).to(torch.bfloat16)
    lp = rq.LoraProjection(w, A, B, torch.ones(2, device=DEV), max_rows=8)
    x, rows = rows_of(8, 512, 32), torch.arange(8, dtype=torch.int32, device=DEV) % 3 - 1
    want = lp(x, rows)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = lp(x, rows, stream=st)
    st.synchronize()
    assert torch.equal(want, y)


def test_graph_replays_with_new_indices(orc):
    """A captured chain replays with the offsets, rows and adapters of the moment."""
    w, What = random_packed(orc, "w4g64", 4 * 96, 256, 33)
    ex = rq.GroupedExperts(w, 4, 32)
    x, off = rows_of(32, 256, 33), torch.zeros(5, dtype=torch.int32, device=DEV)
    y = torch.zeros(32, 96, device=DEV)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        ex(x, off, y=y)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            ex(x, off, y=y)
    for sizes in ([8, 8, 8, 8], [0, 32, 0, 0], [1, 0, 0, 30], [0, 0, 0, 0]):
        o = np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)
        off.copy_(torch.from_numpy(o))
        y.fill_(7.5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        ref = grouped_ref(x, What, 4, o, None)
        if ref:
            rows = sorted(ref)
            check(y[rows], torch.stack([ref[i][0] for i in rows]), torch.stack([ref[i][1] for i in rows]), 256)
        assert (y[int(o[-1]):] == 7.5).all()


def test_chain_as_used(orc):
    """Router, up, channel-mix activation, down, combine: a whole expert layer, captured and replayed."""
    T, C, F, E, k = 21, 256, 512, 8, 2
    up, Wu = random_packed(orc, "w4g64", E * F, C, 34)
    down, Wd = random_packed(orc, "w8g16", E * C, F, 35)
    x = rows_of(T, C, 34)
    logits = torch.randn(T, E, device=DEV)
    logits[5] = -float("inf")                          # a token that the mask leaves without an expert
    gu, gd, router = rq.GroupedExperts(up, E, T * k), rq.GroupedExperts(down, E, T * k), rq.TopkRouter(E, k, renorm=True)

    def layer():
        r = router(logits)
        h = gu(x, r.offsets, in_rows=r.in_rows, act="relu2", out_dtype=torch.bfloat16)
        y = torch.empty(T * k, C, dtype=torch.float32, device=DEV)
        gd(h, r.offsets, out_rows=r.slots, y=y)
        return rq.rq_route_combine(y, r.ids, r.weights), r, h

    out, r, h = layer()
    ids, wts, off = r.ids.cpu().numpy(), r.weights.double(), r.offsets.cpu().numpy()
    assert (ids[5] == -1).all() and off[-1] == (T - 1) * k
    # h against its own formula, then the rest from the h that was used
    rows = r.in_rows.cpu().numpy()
    ref = grouped_ref(x, Wu, E, off, rows)
    live = sorted(ref)
    check(h[live], torch.stack([ref[i][0] for i in live]), torch.stack([ref[i][1] for i in live]), C, act="relu2")
    down_ref = grouped_ref(h, Wd, E, off, None)
    want, S = torch.zeros(T, C, dtype=torch.float64, device=DEV), torch.zeros(T, C, dtype=torch.float64, device=DEV)
    for i in live:
        t, j = divmod(int(r.slots[i]), k)
        want[t] += wts[t, j] * down_ref[i][0]
        S[t] += wts[t, j] * down_ref[i][1]
    check(out, want, S, F + 4 * k)
    assert (out[5] == 0).all()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        layer()
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            again, _, _ = layer()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    assert rq.rq_device_status() == 0
