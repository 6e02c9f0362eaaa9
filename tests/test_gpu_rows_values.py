"""Row-dependent products where a rounding or a range shows: planes made code by
code, so that what a weight is, and what each bound allows, is known exactly.

Bounds (derived): fp32 results are sums of products that are exact in fp32's
range, K 2^-23 sum |x| |w_hat| (an adder that truncates); for the superblocks,
w_hat = S u - M, the two parts are summed apart: K 2^-23 sum |x| (S u + |M|).
bf16 results of many rows come from weights rounded once to fp16: half a step,
2^-11 |w_hat|, or 2^-25 below fp16's normal range; the superblocks' from
S (u - c) + (c S - M), c the middle code, with S, c S - M and the weight rounded
so: 2^-11 (S |u - c| + |c S - M| + |w_hat|) <= 2^-10 (|w_hat| + |c S - M|). A bf16
result adds its own half step, 2^-8.
"""
import numpy as np
import pytest
import torch

import weight_only_quantized_rq_b200 as rq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BITS = {"w4g64": 4, "w8g16": 8, "w8g64": 8, "w6g16": 6, "w4sb32": 4, "w5sb32": 5, "w6sb32": 6}
SYM = ("w4g64", "w8g16", "w8g64", "w6g16")
SB = ("w4sb32", "w5sb32", "w6sb32")


def _pack_bits(v, width):
    """Consecutive `width`-bit fields (last axis) as bytes, lowest bit first."""
    bits = (v[..., None].astype(np.int64) >> np.arange(width)) & 1
    return np.packbits(bits.reshape(*v.shape[:-1], -1).astype(np.uint8), axis=-1, bitorder="little")


def symmetric(fmt, q, s):
    """Packed, w_hat and |w_hat| in 64 bits, from codes q [N][K] and scales s [N][K / group]."""
    N, K = q.shape
    b, s = BITS[fmt], s.astype(np.float16)
    u = (q + 2 ** (b - 1)).astype(np.uint8)
    if fmt == "w4g64":
        codes = _pack_bits(u, 4)
    elif fmt == "w6g16":
        v = u.reshape(N, K // 64, 64)
        codes = np.concatenate((_pack_bits(v & 15, 4), _pack_bits(v >> 4, 2)), -1)
    else:
        codes = u
    _, sb = rq.rq_packed_size(fmt, K, N)
    plane = np.zeros(sb, np.uint8)
    plane[:2 * s.size] = s.reshape(-1).view(np.uint8)
    w = q * np.repeat(s.astype(np.float64), K // s.shape[1], 1)
    return _on_gpu(fmt, K, N, codes, plane, w, np.abs(w))


def superblocks(fmt, u, d, dmin, sc, mn):
    """Packed, w_hat and S u + |M| in 64 bits, from codes u [N][K], d and dmin [N][K / 256], 6-bit sc and mn [N][K / 256][8]."""
    N, K = u.shape
    d, dmin = d.astype(np.float16), dmin.astype(np.float16)
    v = u.reshape(N, K // 256, 256)
    parts = [np.stack((d, dmin), -1).view(np.uint8), _pack_bits(np.concatenate((sc, mn), -1), 6), _pack_bits(v & 15, 4)]
    if BITS[fmt] > 4:
        parts.append(_pack_bits(v >> 4, BITS[fmt] - 4))
    S = np.repeat(d.astype(np.float64)[..., None] * sc, 32, -1).reshape(N, K)
    M = np.repeat(dmin.astype(np.float64)[..., None] * mn, 32, -1).reshape(N, K)
    return _on_gpu(fmt, K, N, np.concatenate(parts, -1), None, S * u - M, S * u + np.abs(M))


def _on_gpu(fmt, K, N, codes, scales, w, size):
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    p = rq.Packed(rq.fmt_id(fmt), K, N, t(codes.reshape(-1)), None if scales is None else t(scales))
    return p, t(w), t(size)


def grouped(w, x, dtype, E=1, sizes=None, **more):
    off = np.concatenate(([0], np.cumsum(sizes if sizes is not None else [x.shape[0]]))).astype(np.int32)
    y = rq.rq_wgemm_grouped(x, w, torch.from_numpy(off).to(DEV), out_dtype=dtype, **more)
    assert rq.rq_device_status() == 0
    return y


def within(y, ref, tol):
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (y.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol.clamp(min=1e-300)).max()))


# Codes that are zero, under scales that are not, at the channels where x is large: what such a channel adds is exactly
# nothing, whatever its size.
def few_codes(fmt, N, K, seed, gone=slice(5, None, 64)):
    """Random codes with zeros at the channels `gone`; no minima for the superblocks (w_hat = S u)."""
    r = np.random.default_rng(seed)
    b = BITS[fmt]
    if fmt in SYM:
        q = r.integers(1 - 2 ** (b - 1), 2 ** (b - 1), (N, K))
        q[:, gone] = 0
        return symmetric(fmt, q, r.uniform(0.5, 1.5, (N, K // (64 if fmt.endswith("g64") else 16))) * 3e-3)
    u = r.integers(0, 2 ** b, (N, K))
    u[:, gone] = 0
    n = (N, K // 256)
    return superblocks(fmt, u, r.uniform(0.5, 1.5, n) * 1e-4, np.zeros(n), r.integers(1, 64, (*n, 8)), r.integers(0, 64, (*n, 8)))


@pytest.mark.parametrize("fmt", SYM + SB)
@pytest.mark.parametrize("M", [1, 8, 15, 40])
@pytest.mark.parametrize("large", [200.0, 3e4])
def test_zero_codes_under_large_activations(fmt, M, large):
    """The same bits as without those channels, and the fp32 bound of the others."""
    K, N = 512, 136
    w, What, _ = few_codes(fmt, N, K, 60 + M)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M))
    x[:, 5::64] *= large
    x = x.to(torch.bfloat16).to(DEV)
    without = x.clone()
    without[:, 5::64] = 0.0
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(grouped(w, x, dtype), grouped(w, without, dtype))
    xd = without.double()
    within(grouped(w, x, torch.float32), xd @ What.t(), K * 2.0 ** -23 * (xd.abs() @ What.abs().t()))


@pytest.mark.parametrize("fmt", SYM + SB)
@pytest.mark.parametrize("M", [1, 12, 40])
def test_all_codes_zero(fmt, M):
    """A matrix of zeros under scales that are not zero gives zeros."""
    K, N = 512, 72
    w, _, _ = few_codes(fmt, N, K, 61, gone=slice(None))
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).to(DEV)
    for dtype in (torch.float32, torch.bfloat16):
        assert (grouped(w, x, dtype) == 0).all()


@pytest.mark.parametrize("fmt", SYM + SB)
@pytest.mark.parametrize("M", [3, 20])
@pytest.mark.parametrize("top", [124, 127])
def test_activations_near_the_largest(fmt, M, top):
    """Finite sums of values up to 2^127: nothing on the way to them leaves fp32's range."""
    K, N = 256, 72
    w, What, _ = few_codes(fmt, N, K, 62)
    keep = 1.0 if top < 127 else 2.0 ** -10               # one channel at the top, the others so that the sums stay finite
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).clamp(-1.9, 1.9).double() * keep
    x[:, 7] = 1.0
    x = (x * 2.0 ** (top - 1)).to(torch.bfloat16).to(DEV)
    xd = x.double()
    y = grouped(w, x, torch.float32)
    assert torch.isfinite(y).all()
    within(y, xd @ What.t(), K * 2.0 ** -23 * (xd.abs() @ What.abs().t()))


@pytest.mark.parametrize("fmt", SYM + SB)
def test_many_rows_round_each_weight_once(fmt):
    """One channel per row, so that each result is one weight: symmetric formats within fp16's half step of it,
    superblocks within 2^-10 of it and of the group's middle weight, also where S u and M nearly cancel."""
    K, N, M = 512, 264, 96
    r = np.random.default_rng(63)
    b, n = BITS[fmt], (N, K // 256)
    if fmt in SYM:
        w, What, _ = few_codes(fmt, N, K, 63, gone=slice(0, 0))
        bound = 2.0 ** -11 * What.abs()
    else:
        d = (r.uniform(0.5, 1.5, n) * 1e-4).astype(np.float16)
        dmin = (d * r.uniform(0.3, 0.7, n) * 2 ** b).astype(np.float16)
        f = lambda: r.integers(48, 64, (*n, 8))
        sc, mn = f(), f()
        w, What, _ = superblocks(fmt, r.integers(0, 2 ** b, (N, K)), d, dmin, sc, mn)
        middle = superblocks(fmt, np.full((N, K), 2 ** (b - 1)), d, dmin, sc, mn)[1]
        bound = 2.0 ** -10 * (What.abs() + middle.abs())
    k = torch.from_numpy(r.permutation(K)[:M]).to(DEV)
    x = torch.zeros(M, K, device=DEV)
    x[torch.arange(M, device=DEV), k] = 2.0 ** torch.randint(-20, 20, (M,), generator=torch.Generator().manual_seed(1)).to(DEV).float()
    x = x.to(torch.bfloat16)
    ref = x.double() @ What.t()
    scale = x.double().sum(1, keepdim=True)
    within(grouped(w, x, torch.bfloat16), ref, x.double() @ bound.t() + 2.0 ** -25 * scale)


def wide_scales(fmt, N, K, seed):
    """Scales over the whole of fp16: a third of the rows ordinary, a third with one huge group, a third huge throughout."""
    r = np.random.default_rng(seed)
    b = BITS[fmt]
    groups = K // (256 if fmt in SB else 64 if fmt.endswith("g64") else 16)
    s = r.uniform(0.5, 1.0, (N, groups)) * 2e-3
    one = np.arange(N) % 3 == 1
    s[one, r.integers(0, groups, int(one.sum()))] = 65504.0
    s[np.arange(N) % 3 == 2] = r.uniform(0.3, 1.0, (int((np.arange(N) % 3 == 2).sum()), groups)) * 65504.0
    if fmt in SYM:
        return symmetric(fmt, r.integers(1 - 2 ** (b - 1), 2 ** (b - 1), (N, K)), s)
    f = lambda: r.integers(0, 64, (N, groups, 8))
    return superblocks(fmt, r.integers(0, 2 ** b, (N, K)), s, s * r.uniform(0.2, 1.0, s.shape), f(), f())


@pytest.mark.parametrize("fmt", SYM + SB)
@pytest.mark.parametrize("M,N,K", [(32, 200, 512), (150, 600, 1024), (700, 130, 256)])
def test_weights_past_half_precision(fmt, M, N, K):
    """Every valid plane gives finite results: weights up to 65504 x 128 (superblocks 65504 x 63 x 64), few and many rows."""
    w, What, size = wide_scales(fmt, 2 * N, K, 64)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).to(DEV)
    xd = x.double()
    h = M // 3
    both = lambda v, W: torch.cat((v[:h] @ W[:N].t(), v[h:] @ W[N:].t()))
    ref, S, F = both(xd, What), both(xd.abs(), What.abs()), both(xd.abs(), size)
    for dtype in (torch.bfloat16, torch.float32):
        tol = K * 2.0 ** -23 * F
        if dtype == torch.bfloat16:
            tol = tol + 2.0 ** -11 * S
        within(grouped(w, x, dtype, sizes=[h, M - h]), ref, tol)
    tol = K * 2.0 ** -23 * F + 2.0 ** -11 * S
    y = grouped(w, x, torch.bfloat16, sizes=[h, M - h], act="relu2")
    within(y, ref.clamp(min=0) ** 2, 2 * ref.abs() * tol + tol * tol + 2.0 ** -23 * ref * ref)


def test_longest_rows_of_weights_past_half_precision():
    """The slow sums of the largest units (128 rows x 256 weight rows x K 32768) end well before any wait gives up."""
    M, N, K = 9500, 150, 32768
    w, What, _ = wide_scales("w8g16", 2 * N, K, 70)
    x = torch.randn(M, K, generator=torch.Generator(device=DEV).manual_seed(70), device=DEV).to(torch.bfloat16)
    y = grouped(w, x, torch.bfloat16, sizes=[M // 2, M // 2])
    for rows, W in ((slice(0, M // 2), What[:N]), (slice(M // 2, M), What[N:])):
        xd = x[rows].double()
        S = xd.abs() @ W.abs().t()
        within(y[rows], xd @ W.t(), (K * 2.0 ** -23 + 2.0 ** -11) * S)


@pytest.mark.parametrize("fmt", ["w4g64", "w8g16", "w6sb32"])
def test_adapters_beside_weights_past_half_precision(fmt):
    M, N, K, r = 70, 200, 512, 16
    w, What, size = wide_scales(fmt, N, K, 65)
    g = torch.Generator().manual_seed(65)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
    A = (torch.randn(3, r, K, generator=g) / K ** 0.5).to(torch.bfloat16).to(DEV)
    B = (torch.randn(3, N, r, generator=g) * 1e3).to(torch.bfloat16).to(DEV)
    a = torch.arange(M, device=DEV) % 3
    xd, Ad, Bd = x.double(), A[a].double(), B[a].double()
    term = torch.einsum("mnr,mrk,mk->mn", Bd, Ad, xd)
    size_t = torch.einsum("mnr,mrk,mk->mn", Bd.abs(), Ad.abs(), xd.abs())
    y = rq.rq_wgemm_lora(x, w, A, B, torch.ones(3, device=DEV), a.to(torch.int32), out_dtype=torch.bfloat16)
    tol = K * 2.0 ** -23 * (xd.abs() @ size.t()) + 2.0 ** -11 * (xd.abs() @ What.abs().t()) + (K + r + 4) * 2.0 ** -23 * size_t
    within(y, xd @ What.t() + term, tol)


@pytest.mark.parametrize("M", [1025, 1030, 1039, 2055])
def test_equal_rows_of_an_adapter_call_are_equal(M):
    """More rows than one round of launches takes, a few left for the last: the call's rows decide how all are multiplied.
    One channel per row (no order of sums), weights of 18 bits, so that a rounding to fp16 in some rows only would show."""
    K, N = 256, 2000
    w, _, _ = few_codes("w8g16", N, K, 66, gone=slice(0, 0))
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    x[:, 77] = 1.0
    g = torch.Generator().manual_seed(66)
    A, B = (torch.randn(1, 8, K, generator=g) / 16).to(torch.bfloat16).to(DEV), torch.randn(1, N, 8, generator=g).to(torch.bfloat16).to(DEV)
    for adapter in (-1, 0):
        rows = torch.full((M,), adapter, dtype=torch.int32, device=DEV)
        y = rq.rq_wgemm_lora(x, w, A, B, torch.ones(1, device=DEV), rows, out_dtype=torch.bfloat16)
        assert (y == y[0]).all(), int((y != y[0]).any(1).sum())
    assert rq.rq_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R", [3, 40])
def test_no_rows_of_x(dtype, R):
    """Indices into an x without rows name no row of it: such rows of the call are rows of zeros, as any other out of range."""
    w, _, _ = few_codes("w4g64", 2 * 40, 256, 67)
    y = torch.full((R + 1, 40), 7.5, dtype=dtype, device=DEV)
    rows = torch.arange(R, dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 1, R - 1], dtype=torch.int32, device=DEV)
    rq.rq_wgemm_grouped(torch.empty(0, 256, dtype=torch.bfloat16, device=DEV), w, off, in_rows=rows - 1, out_rows=rows, y=y[:R])
    assert (y[:R - 1] == 0).all() and (y[R - 1:] == 7.5).all()


def same_infinities(y, ref):
    """Where the formula gives an infinity y has it, where it gives NaN y has NaN."""
    y = y.double()
    assert torch.equal(torch.isnan(y), torch.isnan(ref)), int((torch.isnan(y) != torch.isnan(ref)).sum())
    assert torch.equal(y[torch.isinf(ref)], ref[torch.isinf(ref)])


@pytest.mark.parametrize("fmt", SYM + SB)
@pytest.mark.parametrize("M", [3, 40])
def test_infinite_activations(fmt, M):
    """An infinity beside values of every finite size: its sign with each weight's, NaN where the weight is zero (or, for the
    superblocks' exact products, wherever S u and M are both not zero)."""
    K, N = 256, 72
    w, What, _ = few_codes(fmt, N, K, 68)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(68))
    x[:, 1::3] *= 2.0 ** 100
    x[:, 2::3] *= 2.0 ** -100
    x[0, 9], x[1, 200], x[2, 5] = float("inf"), -float("inf"), float("inf")
    x = x.to(torch.bfloat16).to(DEV)
    ref = x.double() @ What.t()
    for dtype in (torch.float32, torch.bfloat16):
        if fmt in SB and (dtype == torch.float32 or M < 16):
            continue
        same_infinities(grouped(w, x, dtype)[:3], ref[:3])


@pytest.mark.parametrize("M,dtype", [(4, torch.float32), (20, torch.float32), (40, torch.bfloat16)])
def test_infinite_adapters(M, dtype):
    """Infinities in A or B, and a term larger than bf16's largest: the formula's infinities, not NaN."""
    K, N, r = 256, 72, 16
    w, What, _ = few_codes("w8g16", N, K, 69)
    g = torch.Generator().manual_seed(69)
    A = (torch.randn(4, r, K, generator=g) / K ** 0.5).to(torch.bfloat16).to(DEV)
    B = torch.randn(4, N, r, generator=g).to(torch.bfloat16).to(DEV)
    A[0, 3, 17] = float("inf")
    B[1, 40, 5], B[1, 41, 11] = -float("inf"), float("inf")
    A[2] = 0.0
    A[2, 0, 0] = 1.0
    B[2] *= 2.0 ** -20
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
    x[2, 0] = 1.0
    sc = torch.tensor([1.0, 1.0, 3.4e38, 1.0], device=DEV)          # t = 3.4e38 rounds to infinity in bf16, not in fp32
    a = torch.arange(M, device=DEV) % 4
    y = rq.rq_wgemm_lora(x, w, A, B, sc, a.to(torch.int32), out_dtype=dtype)
    xd, Ad, Bd = x.double(), A[a].double(), B[a].double()
    t = (Ad @ xd[..., None]) * sc[a].double()[:, None, None]
    ref = xd @ What.t() + (Bd @ t)[..., 0]
    same_infinities(y[:4], ref[:4])
    assert torch.isfinite(y[[2, 3]]).all()
    within(y[2:3], ref[2:3], 2.0 ** -16 * ref[2:3].abs() + K * 2.0 ** -23 * (xd.abs() @ What.abs().t())[2:3])


@pytest.mark.parametrize("fmt", SYM + SB)
@pytest.mark.parametrize("exp", [-100, -112, -118, -124])
def test_activations_near_the_smallest(fmt, exp):
    """Exact products of values down to 2^-124 and below: codes carry 2^-14, so sums keep fp32's smallest step, 2^-149, times 2^14
    per product of a group (its scale is below 2^-6 here)."""
    K, N, M = 512, 72, 12
    w, What, size = few_codes(fmt, N, K, 71)
    x = (torch.randn(M, K, generator=torch.Generator().manual_seed(71)) * 2.0 ** exp).to(torch.bfloat16).to(DEV)
    xd = x.double()
    y = grouped(w, x, torch.float32)
    within(y, xd @ What.t(), K * 2.0 ** -23 * (xd.abs() @ size.t()) + 2 * K * 2.0 ** -135)
